"""Plain 64-bit forms of the paged-cache operators (append and attention) and a drawn batch."""
import math

import numpy as np
import torch

U = 2.0 ** -24            # half a step of f32, relative
HALF = {"f32": U, "bf16": 2.0 ** -8}
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


class Batch:
    """Sequences given as (new tokens, cached keys before them), their pages drawn at random.

    Pool rows that no sequence or prefix uses, and page-table entries behind a sequence's last
    page, hold NaN and an id outside the pool."""

    def __init__(self, seqs, nq, nkv, hd, page, act="f32", kv="f32", prefix=0, pad=0, seed=0,
                 extra_cols=1):
        r = np.random.default_rng(seed)
        self.nq, self.nkv, self.hd, self.page, self.prefix = nq, nkv, hd, page, prefix
        self.act, self.kv = act, kv
        self.new = np.array([n for n, _ in seqs])
        self.len = np.array([n + p for n, p in seqs])
        self.tokens = int(self.new.sum())
        self.rows = self.tokens + pad
        self.start = np.concatenate([[0], np.cumsum(self.new)])
        pages = -(-self.len // page)
        npre = -(-prefix // page)
        self.n_pages = int(pages.sum()) + npre + 2
        order = r.permutation(self.n_pages)
        self.table = np.full((len(seqs), max(int(pages.max()), 1) + extra_cols), 1 << 30, np.int64)
        at = 0
        for b, n in enumerate(pages):
            self.table[b, :n] = order[at:at + n]
            at += n
        self.pre = order[at:at + npre]
        shape = (self.n_pages, nkv, page, hd)
        self.k = torch.full(shape, math.nan, dtype=DT[kv])
        self.v = torch.full(shape, math.nan, dtype=DT[kv])
        for pool in (self.k, self.v):
            for b in range(len(seqs)):
                for row in range(int(self.len[b])):
                    pool[self.table[b, row // page], :, row % page] = torch.from_numpy(
                        r.standard_normal((nkv, hd))).to(DT[kv])
            for row in range(prefix):
                pool[self.pre[row // page], :, row % page] = torch.from_numpy(
                    r.standard_normal((nkv, hd))).to(DT[kv])
        self.q = torch.from_numpy(r.standard_normal((self.rows, nq, hd)) * 1.5).to(DT[act])
        self.qkv = torch.from_numpy(r.standard_normal((self.rows, (nq + 2 * nkv) * hd))).to(DT[act])

    def cache(self, **kw):
        """The batch on the GPU as a PagedKV."""
        from sequence_decode_step_gb300 import PagedKV

        def ints(a):
            return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()

        self.kd, self.vd = self.k.cuda(), self.v.cuda()
        self.table_d, self.len_d, self.start_d = ints(self.table), ints(self.len), ints(self.start)
        return PagedKV(self.kd, self.vd, self.table_d, self.len_d, self.start_d,
                       prefix_pages=ints(self.pre) if self.prefix else None, prefix_len=self.prefix,
                       **kw)

    def keys(self, pool, b):
        """A sequence's keys behind the prefix, f64 [nkv, prefix + len, hd]."""
        out = []
        for ids, n in ((self.pre, self.prefix), (self.table[b], int(self.len[b]))):
            if n:
                t = pool[torch.from_numpy(np.asarray(ids[:-(-n // self.page)], dtype=np.int64))]
                out.append(t.permute(1, 0, 2, 3).reshape(self.nkv, -1, self.hd)[:, :n])
        if not out:
            return torch.zeros(self.nkv, 0, self.hd, dtype=torch.float64)
        return torch.cat(out, 1).double()

    def attend(self):
        """(output, bound of its error): f64 [tokens, nq, hd] each, rows of no key 0.

        The bound counts, to first order: a score's products and sums (at most hd + 8 roundings of
        the sum of |q k|), the exponential and its argument (2^-22 and the argument's rounding), the
        sums over n keys (at most n / 8 + 64 roundings in a lane, its warp and the joins), and with
        bf16 activations P's rounding; all relative to sum p |v|. Then the output's rounding."""
        g, hd = self.nq // self.nkv, self.hd
        out = torch.zeros(self.tokens, self.nq, hd, dtype=torch.float64)
        tol = torch.zeros_like(out)
        one_term = self.act == "bf16" and self.kv == "bf16"
        for b in range(len(self.new)):
            k, v = self.keys(self.k, b), self.keys(self.v, b)
            for i in range(int(self.new[b])):
                t = int(self.start[b]) + i
                n = self.prefix + int(self.len[b] - self.new[b]) + i + 1
                for h in range(self.nq):
                    kk, vv = k[h // g, :n], v[h // g, :n]
                    q = self.q[t, h].double()
                    s = kk @ q / math.sqrt(hd)
                    p = torch.softmax(s, 0)
                    size = (kk.abs() @ q.abs()).max() / math.sqrt(hd)
                    out[t, h] = p @ vv
                    rel = (hd + 8) * U * size + 4 * U * (s.max() - s.min() + 2) + (n / 8 + 64) * U
                    if one_term:
                        rel = rel + HALF["bf16"]
                    tol[t, h] = 2 * rel * (p @ vv.abs())
        tol += HALF[self.act] * out.abs() + 1e-30
        return out, tol

    def append(self, q_norm=None, k_norm=None, eps=1e-6, theta=1e6, positions=None, sections=None):
        """(q, k rows, v rows, scale): f64, scale = |x_j| + |x_{j+hd/2}| of the rotated heads, which
        bounds a rotation's terms."""
        n, nq, nkv, hd = self.tokens, self.nq, self.nkv, self.hd
        x = self.qkv[:n].double().reshape(n, nq + 2 * nkv, hd)
        q, k, v = x[:, :nq], x[:, nq:nq + nkv], x[:, nq + nkv:]
        if q_norm is not None:
            q = q / (q.pow(2).mean(-1, keepdim=True) + eps).sqrt() * q_norm.double()
            k = k / (k.pow(2).mean(-1, keepdim=True) + eps).sqrt() * k_norm.double()
        half = hd // 2
        f = torch.tensor([theta ** (-2.0 * j / hd) for j in range(half)], dtype=torch.float64)
        if positions is None:
            p = np.concatenate([self.prefix + np.arange(l - m, l) for l, m in zip(self.len, self.new)])
            p = torch.from_numpy(p).double()[:, None].expand(n, half)
        elif sections is None:
            p = positions[:n].double()[:, None].expand(n, half)
        else:
            axis = np.repeat(np.arange(3), sections)
            p = positions[:n].double()[:, torch.from_numpy(axis)]
        z = torch.polar(torch.ones(n, half, dtype=torch.float64), p * f)[:, None]

        def turn(t):
            w = torch.complex(t[..., :half].contiguous(), t[..., half:].contiguous()) * z
            size = (t[..., :half].abs() + t[..., half:].abs())
            return torch.cat([w.real, w.imag], -1), torch.cat([size, size], -1)

        (q, qs), (k, ks) = turn(q), turn(k)
        return q, k, v, qs, ks

    def slots(self):
        """Page and slot of every new token."""
        rows = np.concatenate([np.arange(l - m, l) for l, m in zip(self.len, self.new)])
        seq = np.repeat(np.arange(len(self.new)), self.new)
        return self.table[seq, rows // self.page], rows % self.page
