"""Plain 64-bit forms of the linear layers' activations and the bounds their tests use (CPU)."""
from __future__ import annotations

import math

import torch

import routing_expert_ffn_router_amd as moe

ACTS = {"none": moe.MOE_ACT_NONE, "relu": moe.MOE_ACT_RELU, "silu": moe.MOE_ACT_SILU,
        "gelu": moe.MOE_ACT_GELU, "gelu_tanh": moe.MOE_ACT_GELU_TANH}
DTYPES = {"bf16": (torch.bfloat16, moe.MOE_BF16, 2.0 ** -8),
          "f32": (torch.float32, moe.MOE_F32, 2.0 ** -24)}


def value(z, act):
    if act == "none":
        return z
    if act == "relu":
        return z.clamp(min=0)
    if act == "silu":
        return z * torch.sigmoid(z)
    if act == "gelu":
        return 0.5 * z * torch.erfc(-z / math.sqrt(2))
    return z * torch.sigmoid(math.sqrt(8 / math.pi) * (z + 0.044715 * z ** 3))


def slope(z, act):
    if act == "none":
        return torch.ones_like(z)
    if act == "relu":
        return (z > 0).double()
    if act == "silu":
        s = torch.sigmoid(z)
        return s + z * s * (1 - s)
    if act == "gelu":
        return 0.5 * torch.erfc(-z / math.sqrt(2)) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    c = math.sqrt(8 / math.pi)
    s = torch.sigmoid(c * (z + 0.044715 * z ** 3))
    return s + z * s * (1 - s) * c * (1 + 3 * 0.044715 * z ** 2)


def value_error(z, act):
    """Bound on the fp32 error of act(z) for an exact z.  The functions are within a few units of
    2^-24 (16 allowed here) of |z|; an argument a of exp that is rounded moves it by |a| 2^-24
    of itself, and a e^-a < 1."""
    return 0 * z if act in ("none", "relu") else 16 * 2.0 ** -24 * z.abs()


def slope_error(z, act):
    """... of act'(z): a sum of terms of size 1 and |z| e^-|z| < 1, a few units of 2^-24 each."""
    return 0 * z if act in ("none", "relu") else torch.full_like(z, 16 * 2.0 ** -24)
