"""Bounds that rotated keys in the cache and rotated queries keep to if every token was turned by its own position."""
import torch


def key_bound(want, scale, slack, growths):
    """Codes of the rotated keys `want` (64 bits, off by `slack`) in a block of this scale: half a step of e4m3, 2^-4 of the
    value or 2^-10 scales, and 2^-10 scales more for each time that the scale grew over them."""
    return torch.maximum(2.0 ** -4 * want.abs(), 2.0 ** -10 * scale) + growths * 2.0 ** -10 * scale + 1.07 * slack


def query_bound(want, slack):
    """Half a step of bf16 around what is off by `slack`."""
    return 2.0 ** -8 * want.abs() + 1.01 * slack + 1e-38
