"""Shared helpers of the 8-bit cache tests: caches with known codes, and what
may not be touched filled with bit patterns that would show."""
import numpy as np
import torch

import split_kv_merge_attn_b200 as skv

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}
# half a rounding step relative to the value
HALF_STEP = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11}


def gen(seed):
    return torch.Generator().manual_seed(seed)


def code_values(codes: torch.Tensor) -> np.ndarray:
    """Codes (int8 or e4m3, any device) as float64 values."""
    return codes.cpu().float().double().numpy()


def poisoned_cache(B, Hkv, capacity, D, block, codes):
    """A cache whose every byte is a bad value: e4m3 NaN (0x7f; int8 127) and NaN scales."""
    c = skv.kv8_cache(B, Hkv, capacity, D, block, codes)
    for t in (c.k, c.v):
        t.view(torch.int8).fill_(0x7F)
    for t in (c.k_scale, c.v_scale):
        t.fill_(float("nan"))
    return c


def filled_cache(B, Hkv, capacity, D, block, codes, lengths, seed, scale_span=1.0):
    """Random codes and scales at positions < lengths[b] (whole blocks get a scale),
    bad values behind.  scale_span: the scales' largest power of two."""
    g = gen(seed)
    c = poisoned_cache(B, Hkv, capacity, D, block, codes)
    for codes_t, scale_t in ((c.k, c.k_scale), (c.v, c.v_scale)):
        if codes == "int8":
            x = torch.randint(-127, 128, (B, Hkv, capacity, D), generator=g).to(torch.int8)
        else:
            x = (torch.randn(B, Hkv, capacity, D, generator=g) * 60.0).clamp(-448, 448).to(torch.float8_e4m3fn)
        s = 2.0 ** (scale_span * (torch.rand(B, Hkv, capacity // block, generator=g) - 0.5) - (6 if codes == "int8" else 7))
        for b, n in enumerate(lengths):
            codes_t.view(torch.int8)[b, :, :n] = x.view(torch.int8)[b, :, :n].cuda()
            used = -(-n // block)
            scale_t[b, :, :used] = s[b, :, :used].cuda()
    return c


def values(codes_t, scale_t, lengths):
    """codes * scale in fp64 at positions < lengths[b], 0 behind."""
    x = code_values(codes_t)
    s = scale_t.cpu().double().numpy()
    block = x.shape[2] // s.shape[2]
    out = np.zeros_like(x)
    for b, n in enumerate(lengths):
        out[b, :, :n] = x[b, :, :n] * np.repeat(s[b], block, axis=-1)[:, :n, None]
    return out


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")
