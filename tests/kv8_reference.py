"""Definitions in 64 bits (numpy) of the attention-side operators, block by
block and row by row, and the device tensors of a step for their tests."""
import numpy as np

BLOCK = 16


def bits_to_f64(x):
    """A BF16 torch tensor as float64."""
    return x.detach().float().cpu().numpy().astype(np.float64)


def norm_rotate(x, weight, eps, cos_sin, positions, axis, adjacent):
    """x [t, heads, dim] float64; positions [axes, t] or None (no rotation)."""
    y = x.copy()
    if weight is not None:
        y = y / np.sqrt((y * y).mean(-1, keepdims=True) + eps) * weight
    if cos_sin is None:
        return y
    pairs = cos_sin.shape[1]
    out = y.copy()
    for i in range(pairs):
        row = positions[0 if axis is None else axis[i]]
        c, s = cos_sin[row, i, 0][:, None], cos_sin[row, i, 1][:, None]
        a, b = (2 * i, 2 * i + 1) if adjacent else (i, i + pairs)
        out[..., a] = y[..., a] * c - y[..., b] * s
        out[..., b] = y[..., b] * c + y[..., a] * s
    return out


def attention(q, k, v, n, causal, scale):
    """One sequence: q [n, hq, d], k and v [len, hk, d] -> out, lse, and for
    the tolerances the weights' sum of |v| and the largest sum of |q k|."""
    hq, d = q.shape[1:]
    length, hk = k.shape[:2]
    out, mag = np.zeros((n, hq, d)), np.zeros((n, hq, d))
    lse, reach = np.full((n, hq), -np.inf), np.zeros((n, hq))
    for h in range(hq):
        kh, vh = k[:, h // (hq // hk)], v[:, h // (hq // hk)]
        for i in range(n):
            m = length - n + i + 1 if causal else length
            if m <= 0:
                continue
            s = scale * (kh[:m] @ q[i, h])
            top = s.max()
            p = np.exp(s - top)
            lse[i, h] = top + np.log(p.sum())
            p /= p.sum()
            out[i, h], mag[i, h] = p @ vh[:m], p @ np.abs(vh[:m])
            reach[i, h] = scale * (np.abs(kh[:m]) @ np.abs(q[i, h])).max()
    return out, lse, mag, reach


class Paged:
    """A cache with given sequence lengths in pages in random order; what no
    sequence's token covers holds codes of any value and NaN scales."""

    def __init__(self, lens, heads, dim, page, seed=0, device="cuda", spare=2):
        import torch
        import rotated_int8_quantized_b200 as cr
        g = torch.Generator().manual_seed(seed)
        need = [max(1, -(-n // page)) for n in lens]
        pages = sum(need) + spare
        order = torch.randperm(pages, generator=g).tolist()
        self.table = torch.full((len(lens), max(need) + 1), -1, dtype=torch.int32)
        for b, n in enumerate(need):
            self.table[b, :n] = torch.tensor(order[:n], dtype=torch.int32)
            order = order[n:]
        self.page, self.lens = page, list(lens)
        self.codes, self.scales = [], []
        for _ in "kv":
            c = torch.randint(-127, 128, (pages, heads, page, dim), generator=g, dtype=torch.int8)
            s = torch.full((pages, heads, page // BLOCK), float("nan"))
            for b, n in enumerate(lens):
                for blk in range(-(-n // BLOCK)):
                    p = int(self.table[b, blk * BLOCK // page])
                    s[p, :, blk * BLOCK % page // BLOCK] = (0.5 + torch.rand(heads, generator=g)) / 64
            self.codes.append(c)
            self.scales.append(s)
        self.cache = cr.KV8Cache(*(x.to(device) for x in self.codes + self.scales))
        self.table_dev = self.table.to(device)
        self.kv_len = torch.tensor(lens, dtype=torch.int32, device=device)

    def values(self, b, which, length=None):
        """[length, heads, dim] float64 of sequence b from the device's cache."""
        n = self.lens[b] if length is None else length
        c = (self.cache.k, self.cache.v)[which].cpu().numpy()
        s = (self.cache.k_scale, self.cache.v_scale)[which].cpu().numpy().astype(np.float64)
        at = np.arange(n)
        p, r = self.table.numpy()[b][at // self.page], at % self.page
        return c[p, :, r].astype(np.float64) * s[p, :, r // BLOCK][..., None]
