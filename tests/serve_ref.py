"""Plain 64-bit definitions of the serving operators, for their tests (torch
on the CPU; none of the library's code)."""
import torch

import fp4_block_scaled_quantize_gb300 as fq

HALF_ULP = {torch.bfloat16: 2.0 ** -9, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
# half the spacing of the subnormals: the rounding error of the smallest values
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}

E2M1 = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6],
                    dtype=torch.float64)


def scale_values(kind):
    """Values of the 256 codes of a scale type ("ue5m3", "e4m3", "e8m0")."""
    c = torch.arange(256, dtype=torch.float64)
    if kind == "e8m0":
        return torch.exp2(c - 127)
    if kind == "e4m3":
        c = c % 128
    e, m, bias = torch.floor(c / 8), c % 8, 7 if kind == "e4m3" else 15
    return torch.where(e > 0, (8 + m) * torch.exp2(e - bias - 3), m * 2.0 ** (-2 - bias))


def untile(sf, rows, cols):
    """Scale codes [rows][cols] from the tensor-core layout."""
    c4 = (cols + 3) // 4
    t = sf.view(-1, c4, 32, 4, 4)  # tile row, tile column, line, word, byte
    return t.permute(0, 3, 2, 1, 4).reshape(-1, c4 * 4)[:rows, :cols]


def tile(codes):
    rows, cols = codes.shape
    c4, r128 = (cols + 3) // 4, (rows + 127) // 128
    full = torch.zeros((r128 * 128, c4 * 4), dtype=torch.uint8)
    full[:rows, :cols] = codes
    return full.view(r128, 4, 32, c4, 4).permute(0, 3, 2, 1, 4).contiguous().view(-1)


def weight_values(w):
    """A Quantized copy's values in 64 bits, tensor scale and shifts applied."""
    q, sf = w.q.cpu(), w.sf.cpu()
    n, k = w.rows, w.k
    ue = w.format in (fq.FP4_FMT_UE5M3_B16, fq.FP4_FMT_UE5M3_B32)
    kind = "e8m0" if w.format == fq.FP4_FMT_MXFP4_B32 else "ue5m3" if ue and w.row_shift is None else "e4m3"
    block = 32 if w.format in (fq.FP4_FMT_MXFP4_B32, fq.FP4_FMT_UE5M3_B32) else 16
    if w.sf_layout == fq.FP4_SF_MMA:
        if w.format == fq.FP4_FMT_UE5M3_B32:
            block = 16  # stored once per 16 elements
        codes = untile(sf, n, k // block)
    else:
        codes = sf.view(n, k // block)
    scale = scale_values(kind)[codes.long()]
    if w.row_shift is not None:
        scale = scale * torch.exp2(w.row_shift.cpu()[:n].double())[:, None]
    sd = w.s_dec.cpu().double()
    sd = sd.repeat_interleave(128)[:n] if w.format == fq.FP4_FMT_NVFP4_CTA else sd[:1].expand(n)
    e = E2M1[torch.stack([q & 15, q >> 4], -1).view(n, k).long()]
    return (e.view(n, -1, block) * scale[:, :, None]).view(n, k) * sd[:, None]


def matvec(x, w):
    """(y, sum of magnitudes) in 64 bits."""
    v, x = weight_values(w), x.cpu().double()
    return x @ v.t(), x.abs() @ v.abs().t()


def rotate(x, rope, pos, interleaved):
    """(rotated x, |a cos| + |b sin| per output) for x [T, H, D], float32 rope."""
    x = x.cpu().double()
    y, mag = x.clone(), torch.zeros_like(x)
    if rope is None:
        return y, mag
    r = rope.shape[1]
    cs = rope.cpu().double()[pos.cpu().long().clamp(min=0)]
    co, si = cs[:, None, :r // 2], cs[:, None, r // 2:]
    ia = slice(0, r, 2) if interleaved else slice(0, r // 2)
    ib = slice(1, r, 2) if interleaved else slice(r // 2, r)
    a, b = x[..., ia], x[..., ib]
    y[..., ia], y[..., ib] = a * co - b * si, b * co + a * si
    mag[..., ia], mag[..., ib] = (a * co).abs() + (b * si).abs(), (b * co).abs() + (a * si).abs()
    return y, mag


def attention(q, k_pages, v_pages, table, lengths, scale, window):
    """(out, sum of weighted |v|, lse, largest sum |q k| scale per row), 64 bits."""
    q, kp, vp, table = (t.cpu() for t in (q, k_pages, v_pages, table))
    S, H, D = q.shape
    P, Hk = kp.shape[1], kp.shape[2]
    G = H // Hk
    out, wv = torch.zeros(S, H, D, dtype=torch.float64), torch.zeros(S, H, D, dtype=torch.float64)
    lse, mag = torch.full((S, H), -float("inf"), dtype=torch.float64), torch.zeros(S, H, dtype=torch.float64)
    for s, n in enumerate(lengths.tolist()):
        at = torch.arange(max(0, n - window) if window else 0, n)
        if not len(at):
            continue
        page, place = table[s, at // P].long(), at % P
        k, v = kp[page, place].double(), vp[page, place].double()  # [n, Hk, D]
        qs = q[s].double().view(Hk, G, D)
        score = torch.einsum("kgd,nkd->kgn", qs, k) * scale
        lse[s] = torch.logsumexp(score, -1).reshape(H)
        w = torch.softmax(score, -1)
        out[s] = torch.einsum("kgn,nkd->kgd", w, v).reshape(H, D)
        wv[s] = torch.einsum("kgn,nkd->kgd", w, v.abs()).reshape(H, D)
        mag[s] = (torch.einsum("kgd,nkd->kgn", qs.abs(), k.abs()).amax(-1) * abs(scale)).reshape(H)
    return out, wv, lse, mag
