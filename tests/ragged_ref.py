"""Ragged batches for the tests of paged attention and adapters, and their results in fp64.

The references are the formulas in plain torch fp64, request by request; they share no code with the library."""
from __future__ import annotations

import math

import torch

F64 = torch.float64


def norm_rope(x, w, cos, sin, eps):
    """(n, heads, D): RMSNorm over D with weight (1 + w), then rotation of adjacent pairs."""
    x = x.to(F64)
    x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * (1 + w.to(F64))
    a, b = x[..., 0::2], x[..., 1::2]
    c, s = cos.to(F64)[:, None], sin.to(F64)[:, None]
    return torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2)


class Ragged:
    """Packed new tokens of requests with `new[r]` tokens and kv[r] keys, pages in shuffled order."""

    def __init__(self, d, new, kv, page_size, dtype, device="cpu", spare=0, seed=0, std=1.0):
        g = torch.Generator().manual_seed(seed)
        self.d, self.new, self.kv, self.page_size, self.dtype = d, list(new), list(kv), page_size, dtype
        self.R, self.rows = len(new), sum(new) + spare
        self.start = [0]
        for n in new:
            self.start.append(self.start[-1] + n)
        per = [-(-n // page_size) for n in kv]
        self.num_pages, self.max_pages = sum(per) + 3, max(max(per), 1) + 1
        order = torch.randperm(self.num_pages, generator=g).tolist()
        table = torch.full((self.R, self.max_pages), -1, dtype=torch.int32)
        for r, n in enumerate(per):
            for i in range(n):
                table[r, i] = order.pop()
        KVD = d.Hkv * d.D
        cols = 2 * (d.H + d.Hkv) * d.D

        def rnd(*shape, scale=1.0, dt=dtype):
            return (torch.randn(*shape, generator=g) * scale).to(dt).to(device)

        self.table = table.to(device)
        self.q_start = torch.tensor(self.start, dtype=torch.int32, device=device)
        self.kv_len = torch.tensor(self.kv, dtype=torch.int32, device=device)
        self.qkvg = rnd(self.rows, cols, scale=std)
        self.k_pages, self.v_pages = rnd(self.num_pages, page_size, KVD), rnd(self.num_pages, page_size, KVD)
        self.qw, self.kw = rnd(d.D, scale=0.1, dt=torch.float32), rnd(d.D, scale=0.1, dt=torch.float32)
        angle = torch.rand(self.rows, d.D // 2, generator=g, dtype=F64) * 2 * math.pi
        self.cos, self.sin = torch.cos(angle).float().to(device), torch.sin(angle).float().to(device)

    def slots(self, r, device=None):
        """(page, slot) of every key of request r."""
        t = torch.arange(self.kv[r], device=self.table.device)
        return self.table[r].long()[t // self.page_size], t % self.page_size

    def rowsof(self, r):
        return slice(self.start[r], self.start[r + 1])

    def poison(self, value=float("nan")):
        """Fills everything that no key of the batch occupies with `value`."""
        keep = torch.zeros(self.num_pages, self.page_size, dtype=torch.bool, device=self.table.device)
        for r in range(self.R):
            p, s = self.slots(r)
            keep[p, s] = True
        self.k_pages[~keep] = value
        self.v_pages[~keep] = value

    def appended(self):
        """k_pages, v_pages in fp64 after the append."""
        d = self.d
        k, v = self.k_pages.to(F64), self.v_pages.to(F64)
        for r in range(self.R):
            n, sl = self.new[r], self.rowsof(r)
            if n == 0:
                continue
            p, s = self.slots(r)
            x = self.qkvg[sl]
            kk = norm_rope(x[:, d.HD:d.HD + d.KVD].reshape(n, d.Hkv, d.D), self.kw, self.cos[sl], self.sin[sl], d.eps)
            k[p[-n:], s[-n:]] = kk.reshape(n, d.KVD)
            v[p[-n:], s[-n:]] = x[:, d.HD + d.KVD:d.HD + 2 * d.KVD].to(F64)
        return k, v

    def attention(self, text_mask=None, key_end=None, k_pages=None, v_pages=None):
        """(rows, H*D) in fp64, and sigmoid(g) sum_k p_k |v_k|, the size that errors of the probabilities are
        relative to; rows behind the last request are NaN."""
        d = self.d
        out = torch.full((self.rows, d.HD), float("nan"), dtype=F64, device=self.qkvg.device)
        size = out.clone()
        kp, vp = (self.k_pages if k_pages is None else k_pages), (self.v_pages if v_pages is None else v_pages)
        for r in range(self.R):
            n, L, sl = self.new[r], self.kv[r], self.rowsof(r)
            if n == 0:
                continue
            p, s = self.slots(r)
            x = self.qkvg[sl]
            q = norm_rope(x[:, :d.HD].reshape(n, d.H, d.D), self.qw, self.cos[sl], self.sin[sl], d.eps)
            seen = torch.ones(n, L, dtype=torch.bool, device=q.device)
            if text_mask is not None:
                T = min(text_mask.shape[1], L)
                seen[:, :T] &= text_mask[r, :T].bool()
            if key_end is not None:
                low = torch.arange(L - n + 1, L + 1, device=q.device)
                end = torch.maximum(key_end[sl].long(), low).clamp(max=L)
                seen &= torch.arange(L, device=q.device)[None] < end[:, None]
            k = kp[p, s].to(F64).reshape(L, d.Hkv, d.D)
            v = vp[p, s].to(F64).reshape(L, d.Hkv, d.D)
            any_seen = seen.any(0)[:, None, None]
            k, v = torch.where(any_seen, k, 0.0), torch.where(any_seen, v, 0.0)
            g = torch.sigmoid(x[:, d.HD + 2 * d.KVD:].to(F64)).reshape(n, d.H, d.D)
            for h in range(d.H):
                j = h // (d.H // d.Hkv)
                z = (q[:, h] @ k[:, j].T / math.sqrt(d.D)).masked_fill(~seen, -math.inf)
                top = z.amax(1, keepdim=True)
                w = torch.exp(z - torch.where(top == -math.inf, 0.0, top))
                total = w.sum(1, keepdim=True)
                o = torch.where(total > 0, w @ v[:, j] / torch.where(total > 0, total, 1.0), 0.0)
                a = torch.where(total > 0, w @ v[:, j].abs() / torch.where(total > 0, total, 1.0), 0.0)
                out[sl, h * d.D:(h + 1) * d.D] = o * g[:, h]
                size[sl, h * d.D:(h + 1) * d.D] = a * g[:, h]
        return out, size


def lora_ref(A, W, down, up, scale, start, ids, epilogue, out0=None, gate=None, rows_per_batch=0):
    """y of every row that belongs to a request, in fp64; other rows keep out0 (fp64)."""
    res = out0.to(F64).clone()
    for r in range(len(ids)):
        a, b = start[r], start[r + 1]
        if a == b:
            continue
        x = A[a:b].to(F64)
        y = x @ W.to(F64).T
        j = ids[r]
        if j >= 0:
            y = y + scale[j].to(F64) * ((x @ down[j].to(F64).T) @ up[j].to(F64).T)
        if epilogue == "swiglu":
            y = y.reshape(b - a, -1, 2, 64)
            y = (y[:, :, 0] * torch.sigmoid(y[:, :, 0]) * y[:, :, 1]).reshape(b - a, -1)
        if epilogue == "resid":
            rows = torch.arange(a, b, device=A.device)
            gr = gate[rows // rows_per_batch] if rows_per_batch else gate[r].expand(b - a, -1)
            y = res[a:b] + gr.to(F64) * y
        res[a:b] = y
    return res


def off(got, ref):
    """(2-norm of the error over the 2-norm of ref, largest error over max(rms, |ref|))."""
    got, ref = got.to(F64), ref.to(F64)
    err = got - ref
    rms = ref.square().mean().sqrt().clamp(min=1e-300)
    rel = float(err.square().mean().sqrt() / rms)
    big = float((err.abs() / torch.maximum(ref.abs(), rms)).max())
    print(f"rel {rel:.3e} max {big:.3e}")
    return rel, big
