"""MXFP4 in plain 64-bit torch: the definition, apart from the kernels' code."""
import torch

F64 = torch.float64
MAGNITUDES = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=F64)


def power(e):
    """2 ** e in 64 bits, from its bits (pow of the GPU's library is not exact)."""
    return (e.to(torch.int64) + 1023 << 52).view(F64)


def quant(x):
    """(codes, scales) of x [..., rows, D] by searching the eight magnitudes:
    the nearest, of two the one with an even code."""
    v = x.detach().cpu().to(F64).unflatten(-1, (-1, 32))
    top = v.abs().amax(-1)
    bad = ~torch.isfinite(top)
    _, e = torch.frexp(torch.where(bad | (top == 0), 1.0, top))   # top = m * 2^e, m in 0.5 .. 1
    s = (e - 3 + 127).clamp(min=0)
    s = torch.where(top == 0, 0, torch.where(bad, 255, s))
    r = torch.where(bad[..., None], 0.0, v.abs()) * power(127 - s.to(torch.int64))[..., None]
    far = (r.clamp(max=6.0)[..., None] - MAGNITUDES).abs()
    far = 2 * far / far.amin(-1, keepdim=True).clamp(min=1e-300)  # exact for ties
    code = (far + torch.arange(8) % 2 * 1e-9).argmin(-1)
    code = torch.where(bad[..., None], 0, code + 8 * torch.signbit(v))
    code = code.to(torch.uint8).flatten(-2)
    s = torch.nn.functional.pad(s.to(torch.uint8), (0, -s.shape[-1] % 4))
    s = s.unflatten(-1, (-1, 4)).transpose(-2, -3).contiguous()
    return code[..., ::2] | code[..., 1::2] << 4, s


def values(codes, scales):
    """[..., rows, D] in 64 bits, on the tensors' device."""
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).long()
    v = MAGNITUDES.to(c.device)[c & 7] * (1.0 - 2.0 * (c >> 3))
    s = scales.transpose(-2, -3).flatten(-2)
    p = torch.where(s == 255, float("nan"), power(s.to(torch.int64) - 127))
    return v * p.repeat_interleave(32, -1)[..., :v.shape[-1]]


def random(shape, seed, device="cuda", low=120, high=126):
    """Random codes and scales of a [.., rows, D] tensor."""
    g = torch.Generator(device=device).manual_seed(seed)
    *lead, rows, D = shape
    codes = torch.randint(0, 256, (*lead, rows, D // 2), generator=g, device=device, dtype=torch.uint8)
    scales = torch.randint(low, high + 1, (*lead, -(-D // 128), rows, 4), generator=g, device=device,
                           dtype=torch.uint8)
    if D % 128:
        scales[..., -1, :, D % 128 // 32:] = 0
    return codes, scales
