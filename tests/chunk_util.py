"""Plain 64-bit forms of the chunk operators (rotated append, attention of a chunk of new
tokens), random ragged batches for them, and the tolerances their roundings allow."""

import math

import torch

HEADS, DIM = 64, 256
F64 = torch.float64


# ---------------------------------------------------------------------- plain forms


def rotate(x, cos, sin, interleaved):
    """x [T, ..., 256] float64; cos, sin [T, P]: pair i of the first 2 P dimensions turned by
    the token's angle i."""
    p = cos.shape[1]
    shape = [x.shape[0]] + [1] * (x.dim() - 2) + [p]
    c, s = cos.reshape(shape), sin.reshape(shape)
    y = x.clone()
    one = torch.arange(p) * 2 if interleaved else torch.arange(p)
    two = one + 1 if interleaved else one + p
    a, b = x[..., one], x[..., two]
    y[..., one] = a * c - b * s
    y[..., two] = b * c + a * s
    return y


def angles(table, rot_dim, pair_axis, positions):
    """cos, sin [T, P] of positions [axes, T]."""
    p = rot_dim // 2
    pos = torch.stack([positions[a].long() for a in pair_axis], 1)  # [T, P]
    i = torch.arange(p, device=table.device)
    return table[pos, i].to(F64), table[pos, p + i].to(F64)


def attention(q, k, v, first, scale):
    """q [n, 64, 256] float64 of positions first .. first + n - 1, k and v [L, 256] float64:
    (out; for the tolerance: the same of |V|, and the largest weight times the sum of |V|)."""
    n, length = q.shape[0], k.shape[0]
    s = torch.einsum("nhd,ld->nhl", q, k) * scale
    seen = torch.arange(length, device=q.device)[None] <= \
        first + torch.arange(n, device=q.device)[:, None]
    s = torch.where(seen[:, None], s, torch.full_like(s, -math.inf))
    p = torch.softmax(s, -1)
    # (a hidden row's values do not take part, whatever they are)
    out = torch.empty(n, HEADS, DIM, dtype=F64, device=q.device)
    mag, top = torch.empty_like(out), torch.empty_like(out)
    for i in range(n):
        end = first + i + 1
        out[i] = p[i, :, :end] @ v[:end]
        mag[i] = p[i, :, :end] @ v[:end].abs()
        top[i] = p[i].amax(-1, keepdim=True) * v[:end].abs().sum(0)
    return out, mag, top


# ---------------------------------------------------------------------- ragged batches


class Batch:
    """A ragged batch: n[b] new tokens after c[b] cached positions, K and V of all of them in a
    contiguous (page 0) or paged cache of bf16 or e4m3 values. Rows past a sequence's end hold
    `tail` (e.g. NaN)."""

    def __init__(self, new, cached, fp8=False, page=0, seed=0, spare=0, tail=None, lead=0,
                 behind=0, q_scale=1.0, device="cuda"):
        g = torch.Generator().manual_seed(seed)
        self.new, self.cached = list(new), list(cached)
        self.total = [a + b for a, b in zip(new, cached)]
        self.batch, self.fp8, self.page = len(new), fp8, page
        self.k_scale, self.v_scale = (0.011, 0.013) if fp8 else (1.0, 1.0)
        self.lead = lead
        starts = [lead]
        for x in new:
            starts.append(starts[-1] + x)
        self.starts, self.rows = starts, starts[-1] + behind
        dev = torch.device(device)
        self.dev = dev
        self.q = (torch.randn(max(1, self.rows), HEADS, DIM, generator=g) * q_scale).to(
            torch.bfloat16).to(dev)
        self.q_start = torch.tensor(starts, dtype=torch.int32, device=dev)
        self.seq_lens = torch.tensor(self.total, dtype=torch.int32, device=dev)
        dt = torch.float8_e4m3fn if fp8 else torch.bfloat16

        def store(x, s):
            return (x / s).clamp(-448, 448).to(dt) if fp8 else x.to(dt)

        kv = [[store(torch.randn(max(t, 1), DIM, generator=g), s) for t in self.total]
              for s in (self.k_scale, self.v_scale)]
        self.cap = [max(t, 1) + spare for t in self.total]
        if page:
            per = [-(-c // page) for c in self.cap]
            self.per_seq = per
            pool = sum(per) + 2
            order = torch.randperm(pool, generator=g)
            self.table = torch.zeros(self.batch, max(per), dtype=torch.int32)
            bufs = [torch.empty(pool, page, DIM, dtype=dt) for _ in range(2)]
            for buf in bufs:
                _fill(buf, tail)
            at = 0
            for b in range(self.batch):
                ids = order[at:at + per[b]]
                at += per[b]
                self.table[b, :per[b]] = ids.to(torch.int32)
                for buf, src in zip(bufs, kv):
                    for j in range(-(-self.total[b] // page)):
                        rows = src[b][j * page:min((j + 1) * page, self.total[b])]
                        _bits(buf)[ids[j], :rows.shape[0]] = _bits(rows)
            self.table = self.table.to(dev)
            self.k, self.v = (t.to(dev) for t in bufs)
        else:
            out = []
            for src in kv:
                seqs = []
                for b in range(self.batch):
                    t = torch.empty(self.cap[b], DIM, dtype=dt)
                    _fill(t, tail)
                    _bits(t)[:self.total[b]] = _bits(src[b])[:self.total[b]]
                    seqs.append(t.to(dev))
                out.append(seqs)
            self.k, self.v = out

    def cache(self):
        from decode_attention_10_b200 import mfa
        if self.page:
            return mfa.PagedKVCache(self.k, self.v, self.table, self.per_seq, self.k_scale,
                                    self.v_scale)
        return mfa.KVCache(self.k, self.v, self.k_scale, self.v_scale)

    def stored(self, which, b, rows=None):
        """The stored K or V rows of sequence b (as the cache's type)."""
        rows = self.total[b] if rows is None else rows
        buf = self.k if which == "k" else self.v
        if not self.page:
            return buf[b][:rows]
        ids = self.table[b].tolist()[:-(-rows // self.page)]
        t = torch.cat([_bits(buf)[i] for i in ids]) if ids else _bits(buf)[0][:0]
        return t[:rows].view(buf.dtype)

    def values(self, which, b):
        s = self.k_scale if which == "k" else self.v_scale
        return self.stored(which, b).to(F64) * s

    def reference(self, scale=1.0 / 16.0):
        """(out, tolerance) [rows, 64, 256] float64; NaN out where a row is nobody's."""
        out = torch.full((self.rows, HEADS, DIM), math.nan, dtype=F64, device=self.dev)
        tol = torch.zeros_like(out)
        for b in range(self.batch):
            if self.new[b] == 0:
                continue
            rows = slice(self.starts[b], self.starts[b + 1])
            q = self.q[rows].to(F64)
            k, v = self.values("k", b), self.values("v", b)
            o, mag, top = attention(q, k, v, self.cached[b], scale)
            out[rows] = o
            # one rounding of the result (half a bf16 step: 2^-8 of it); the weights rounded
            # to bf16, or to an e4m3 pair within 2^-8 of them; a score's 256 products are
            # summed in float32 (256 steps of at most 2^-23 each of their magnitudes' sum:
            # the tensor core may truncate), which moves a weight by twice that at most
            dot = torch.einsum("nhd,ld->nhl", q.abs(), k.abs()).amax(-1, keepdim=True)
            score = 256 * 2.0 ** -23 * dot * scale
            if self.fp8:
                # q as an e4m3 pair: exact within 2^-10 of the row's largest, half the
                # smallest step of the low part (2^-10 of a largest of at least 128) below
                qmax = q.abs().amax(-1, keepdim=True)
                score = score + 2.0 ** -17 * qmax * k.abs().sum(-1).max() * scale
                # a weight p is the e4m3 pair of 2^(s - m + 4), m at most the row's largest
                # score: the largest is 2^4 or more. A pair is off by at most half a step of
                # its low part: 2^-8 of p, or, where that is subnormal, half of 2^-9, which is
                # at most 2^-14 of the largest weight
                mag = mag + 2.0 ** -6 * top
            tol[rows] = 2.0 ** -8 * o.abs() + (2.0 ** -8 + 2 * score) * mag + 1e-30
        return out, tol


def _bits(t):
    return t.view(torch.uint8 if t.element_size() == 1 else torch.int16)


def _fill(t, tail):
    if tail is None:
        _bits(t).zero_()
    elif t.element_size() == 1:
        _bits(t).fill_(0x7F)  # the e4m3 NaN (it has no infinity)
    else:
        t.fill_(tail)


def check(got, batch, ref=None, scale=1.0 / 16.0):
    out, tol = batch.reference(scale) if ref is None else ref
    rows = ~out.isnan().all(-1).all(-1)
    d = (got.to(F64) - out).abs()[rows]
    bad = ~(d <= tol[rows])
    if bad.any():
        at = bad.nonzero()[0].tolist()
        raise AssertionError(f"{int(bad.sum())} of {bad.numel()} elements off; first at {at}: "
                             f"off by {float(d[tuple(at)]):.3e}, may be "
                             f"{float(tol[rows][tuple(at)]):.3e}; largest {float(d.max()):.3e}")
