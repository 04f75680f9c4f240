"""Inputs and tolerances shared by the tests of the attention side (norm and rotation, 4-bit cache,
sparse attention)."""
import numpy as np

import workloads as W
from oracle import attention as A


def round_to(x, f16):
    """float32 values of x rounded to float16, or truncated to bfloat16."""
    x = np.ascontiguousarray(x, np.float32)
    if f16:
        return x.astype(np.float16).astype(np.float32)
    return (x.view(np.uint32) & np.uint32(0xFFFF0000)).view(np.float32)


def half_step(f16):
    """Largest relative rounding error of the type: half a step, eps / 2."""
    return 2.0 ** -11 if f16 else 2.0 ** -8


def smallest_step(f16):
    """Half the spacing of the type's subnormals (an absolute rounding error below its normal range)."""
    return 2.0 ** -25 if f16 else 2.0 ** -134


def table(max_pos, rotary, base=10000.0):
    ang = np.arange(max_pos)[:, None] * base ** (-np.arange(0, rotary, 2) / max(rotary, 1))[None, :]
    return np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)


def cache_case(**kw):
    """A workload whose block_table and lengths the KV cache shares."""
    return W.make_case("kv", **kw)


def cache(case, heads, dim, e2m1, seed, k_scale=1.0, v_scale=1.0):
    """A pool uint8 [num_blocks, block_size, entry_bytes]: quantised normal keys and values of spread-out
    magnitudes in every slot, random padding bytes."""
    rng = np.random.default_rng(seed)
    n = case.num_blocks * case.block_size
    k = rng.normal(size=(n, heads, dim)) * np.exp(rng.uniform(-2, 1, size=(n, heads, 1))) * k_scale
    v = rng.normal(size=(n, heads, dim)) * np.exp(rng.uniform(-2, 1, size=(n, heads, 1))) * v_scale
    junk = rng.integers(0, 256, size=(n, A.entry_bytes(heads, dim)), dtype=np.uint8)
    e = A.encode(k.astype(np.float32), v.astype(np.float32), e2m1, k_scale, v_scale, into=junk)
    return e.reshape(case.num_blocks, case.block_size, -1)


def attention_bounds(ref, lse, spread, dim, f16):
    """Derived bounds of |out - ref| and |lse - ref| for: queries within 2^-25 of their head's largest
    magnitude, exact keys and values, fp32 logits and accumulators (each of the D or n additions of a
    product sum within 2^-23 of the sum of magnitudes, truncation allowed), an exponential within
    2^-21, probabilities rounded to fp16 (2^-11 relative, 2^-25 absolute below its normal range, of a
    largest probability of at least 1), one rounding of the output."""
    n = np.maximum(spread["n"], 1)[:, None]
    dz = spread["qk"] * (dim + 16) * 2.0 ** -23 * 2 + spread["kq"] * 2.0 ** -25
    rel = 2.0 ** -11 + 2 * dz + (n + 64) * 2.0 ** -23 + 2.0 ** -20
    err = rel[..., None] * (spread["wv"] + np.abs(ref)) + (n * 2.0 ** -25 * spread["vmax"])[..., None]
    tol = err + half_step(f16) * (np.abs(ref) + err) + smallest_step(f16)
    return tol, dz + 2.0 ** -20 + n * 2.0 ** -23 + 2.0 ** -22 * np.where(np.isfinite(lse), np.abs(lse), 0)
