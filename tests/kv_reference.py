"""The paged 4-bit cache in 64 bits, from its definition: quantising, reading, rotating,
attending.  Plain loops over sequences; nothing of the library's."""
import math

import torch

E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def nearest(x, grid):
    """x >= 0 (a number) to the nearest of an ascending grid, ties to its even places."""
    x = min(max(x, 0.0), grid[-1])
    hi = next(i for i, v in enumerate(grid) if v >= x)
    if hi == 0:
        return 0
    a, b = x - grid[hi - 1], grid[hi] - x
    return hi - 1 if a < b or (a == b and hi % 2 == 1) else hi


def e4m3_grid():
    return [float(v) for v in torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).float()]


_E4M3 = e4m3_grid()


def quantise(y, head_scale=1.0):
    """16 numbers -> (codes, scale's byte)."""
    if any(math.isnan(v) for v in y):
        return [0] * 16, 0x7F
    top = max(abs(v) for v in y)
    byte = nearest(top / (6.0 * head_scale), _E4M3)
    s = _E4M3[byte] * head_scale
    if byte == 0:
        return [0] * 16, 0
    return [nearest(abs(v) / s, E2M1) | (8 if v < 0 else 0) for v in y], byte


def decode(cache, page_size, head_dim):
    """[pages][heads][2][page_size][head_dim] in FP64, without the heads' scales."""
    n = page_size * head_dim // 2
    codes = cache[..., :n].unflatten(-1, (page_size, head_dim // 2)).int()
    codes = torch.stack([codes & 15, codes >> 4], -1).flatten(-2)
    table = torch.tensor(E2M1 + [-v for v in E2M1], dtype=torch.float64, device=cache.device)
    scales = cache[..., n:].contiguous().view(torch.float8_e4m3fn).double()
    scales = scales.unflatten(-1, (page_size, head_dim // 16)).repeat_interleave(16, -1)
    return table[codes.long()] * scales


def sequences(cu, kv_lens, T):
    """(first row, rows, length) of every sequence; cu None: rows evenly."""
    n = len(kv_lens)
    if cu is None:
        cu = [i * (T // n) for i in range(n + 1)]
    out = []
    for i in range(n):
        b, e = cu[i], cu[i + 1]
        out.append((b, e - b if 0 <= b <= e <= T else 0, kv_lens[i]))
    return out


def page_of(table, s, at, page_size, n_pages):
    if at < 0 or at >= table.shape[1] * page_size:
        return None
    page = int(table[s, at // page_size])
    return page if 0 <= page < n_pages else None


def rotate(x, positions, inv_freq, interleaved):
    """x [T][heads][D] in FP64, its first 2 len(inv_freq) elements turned."""
    x = x.double().clone()
    half = inv_freq.shape[0]
    if half == 0:
        return x
    angle = positions.double()[:, None, None] * inv_freq.double()
    c, s = torch.cos(angle), torch.sin(angle)
    if interleaved:
        a, b = x[..., 0:2 * half:2].clone(), x[..., 1:2 * half:2].clone()
        x[..., 0:2 * half:2], x[..., 1:2 * half:2] = a * c - b * s, b * c + a * s
    else:
        a, b = x[..., :half].clone(), x[..., half:2 * half].clone()
        x[..., :half], x[..., half:2 * half] = a * c - b * s, b * c + a * s
    return x


def attention(q, cache, table, kv_lens, page_size, cu=None, k_scale=None, v_scale=None, scale=None, causal=True,
              window=0):
    """(out, lse, spread, size): out and lse in FP64 (rows of no sequence NaN); spread [T][H][D] = sum p |v|, what
    a relative error of p is relative to; size [T][H] = the largest sum |q_i k_i| scale of a seen token."""
    T, H, D = q.shape
    G = cache.shape[1]
    dev = q.device
    out = torch.full((T, H, D), math.nan, dtype=torch.float64, device=dev)
    spread = out.clone()
    lse, size = (torch.full((T, H), math.nan, dtype=torch.float64, device=dev) for _ in range(2))
    scale = D ** -0.5 if scale is None else scale
    table_c = table.cpu()
    lens = [int(v) for v in kv_lens]
    for s, (row, n, length) in enumerate(sequences(None if cu is None else [int(v) for v in cu], lens, T)):
        if n == 0:
            continue
        held = max(0, min(length, table_c.shape[1] * page_size))
        pages = [page_of(table_c, s, j, page_size, cache.shape[0]) for j in range(0, held, page_size)]
        there = torch.tensor([p is not None for p in pages], dtype=torch.bool, device=dev).repeat_interleave(page_size)[:held]
        at = torch.tensor([p or 0 for p in pages], dtype=torch.long, device=dev)
        kv = decode(cache[at], page_size, D)  # [pages][G][2][page][D]
        place = torch.arange(length - n, length, device=dev)[:, None]
        j = torch.arange(held, device=dev)[None]
        seen = there[None] & (j <= place if causal else j >= 0)
        if window:
            seen = seen & (j > place - window)
        for g in range(G):
            k = kv[:, g, 0].reshape(-1, D)[:held] * (1.0 if k_scale is None else float(k_scale[g]))
            v = kv[:, g, 1].reshape(-1, D)[:held] * (1.0 if v_scale is None else float(v_scale[g]))
            bad = v.isnan().any(-1)  # makes a row that sees it NaN
            v = v.masked_fill(bad[:, None], 0.0)
            x = q[row:row + n, g::G].double()  # [n][r][D]
            z = x @ k.T * scale
            z = torch.where(bad, math.nan, z)
            z = torch.where(seen[:, None], z, -math.inf)
            top = z.amax(-1, keepdim=True) if held else torch.full((n, x.shape[1], 1), -math.inf, device=dev)
            p = torch.exp(z - torch.where(top == -math.inf, 0.0, top))
            total = p.sum(-1, keepdim=True)
            some = total != 0  # (NaN is)
            out[row:row + n, g::G] = torch.where(some, (p @ v) / total, 0.0)
            spread[row:row + n, g::G] = torch.where(some, (p @ v.abs()) / total, 0.0)
            lse[row:row + n, g::G] = torch.where(some, top + total.log(), -math.inf)[..., 0]
            if held:
                big = x.abs() @ k.nan_to_num(0.0).abs().T * abs(scale)
                size[row:row + n, g::G] = torch.where(seen[:, None], big, 0.0).amax(-1)
            else:
                size[row:row + n, g::G] = 0
    return out, lse, spread, size
