"""The measured cases of the chunk operators: appending rotated keys and values to a KV cache
(with the query rotation of the same tokens, positions on one or several axes), and the
attention of a chunk of new tokens over the cache.

Both take a ragged batch: sequence b owns rows q_start[b] .. q_start[b + 1] of the new tokens
(64 query heads of 256, one shared K and one shared V head), the last n_b of its seq_lens[b]
cached positions. `run` makes the framework's calls where `own` is true, and computes the same
in elementary torch operations (float32, rounded once at the end) where it is false.
"""

import math
import random

import torch

own = False

HEADS, DIM = 64, 256
SCALE = 1.0 / 16.0
MAX_POS = 65536
# score elements of one batched product of the plain attention (16 GiB in float32)
SCORES = 1 << 32


def listed():
    return [
        # the tail of a short prompt, or three drafted tokens checked: launch latency
        dict(name="attn_bf16_1x3_l130", op="attn", kv="bf16", page=64, batch=1, n_lo=3, n_hi=3,
             c_lo=127, c_hi=127, lens=1),
        # a serving step that decodes one token a sequence through the chunk call
        dict(name="attn_bf16_32x1_l4096", op="attn", kv="bf16", page=128, batch=32, n_lo=1,
             n_hi=1, c_lo=4095, c_hi=4095, lens=2),
        # speculative decoding: four drafted tokens a sequence, contiguous buffers
        dict(name="attn_bf16_32x4_l4096", op="attn", kv="bf16", page=0, batch=32, n_lo=4,
             n_hi=4, c_lo=4092, c_hi=4092, lens=3),
        # a whole prompt of odd length, nothing cached before
        dict(name="attn_bf16_1x1111_l1111", op="attn", kv="bf16", page=64, batch=1, n_lo=1111,
             n_hi=1111, c_lo=0, c_hi=0, lens=4),
        # a chunk of a prompt of 8192 tokens
        dict(name="attn_bf16_1x2048_l8192", op="attn", kv="bf16", page=128, batch=1, n_lo=2048,
             n_hi=2048, c_lo=6144, c_hi=6144, lens=5),
        # the last chunk of the longest context
        dict(name="attn_bf16_1x509_l65536", op="attn", kv="bf16", page=256, batch=1, n_lo=509,
             n_hi=509, c_lo=65027, c_hi=65027, lens=6),
        # continuous batching: decoding sequences and prompt chunks in one call, FP8 pages
        dict(name="attn_fp8_24mixed", op="attn", kv="fp8", page=64, batch=24, n_lo=1, n_hi=700,
             c_lo=100, c_hi=9000, lens=7),
        # two prompt chunks over FP8 buffers
        dict(name="attn_fp8_2x1500_l6000", op="attn", kv="fp8", page=0, batch=2, n_lo=1500,
             n_hi=1500, c_lo=4500, c_hi=4500, lens=8),
        # the append of a decoding step: launch latency
        dict(name="append_bf16_32x1", op="append", kv="bf16", page=128, batch=32, n_lo=1,
             n_hi=1, c_lo=200, c_hi=4000, lens=9, rot=256, pairing="halves", axes=1),
        # the append of a batch of prompt chunks
        dict(name="append_bf16_5x1700", op="append", kv="bf16", page=64, batch=5, n_lo=1500,
             n_hi=1900, c_lo=0, c_hi=4000, lens=10, rot=256, pairing="halves", axes=1),
        # decoding next to a video: three axes, half of the dimensions rotated, FP8 cache
        dict(name="append_fp8_64x1_video", op="append", kv="fp8", page=0, batch=64, n_lo=1,
             n_hi=1, c_lo=100, c_hi=3000, lens=11, rot=128, pairing="neighbours", axes=3),
        # the tokens of a video (time, height, width) appended to FP8 pages
        dict(name="append_fp8_1x5001_video", op="append", kv="fp8", page=128, batch=1,
             n_lo=5001, n_hi=5001, c_lo=77, c_hi=77, lens=12, rot=256, pairing="halves",
             axes=3),
    ]


def _log_int(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm (0 counted as 1/2)."""
    a, b = math.log(max(lo, 0.5)), math.log(hi + 0.999)
    return max(lo, min(hi, int(math.exp(rng.uniform(a, b)))))


def draw(rng):
    page = rng.choice([0, 64, 128, 256, 512])
    kv = rng.choice(["bf16", "fp8"])
    lens = rng.randrange(1 << 30)
    append = rng.random() < 0.4
    while True:
        batch = _log_int(rng, 1, 64 if append else 48)
        if append:
            n_hi = _log_int(rng, 1, 8000 // batch)
            c_hi = _log_int(rng, 1, 8000)
            case = dict(op="append", kv=kv, page=page, batch=batch,
                        n_lo=rng.choice([0, 1, (n_hi + 1) // 2]), n_hi=n_hi, c_lo=c_hi // 4,
                        c_hi=c_hi, lens=lens, rot=rng.choice([64, 128, 192, 256]),
                        pairing=rng.choice(["halves", "neighbours"]),
                        axes=rng.choice([1, 1, 2, 3]))
            if sum(_lens(case)[0]):
                return case
            continue
        n_hi = _log_int(rng, 1, 2048)
        c_hi = rng.choice([0, *(_log_int(rng, 30, 60000) for _ in range(6))])
        case = dict(op="attn", kv=kv, page=page, batch=batch,
                    n_lo=rng.choice([0, 1, (n_hi + 1) // 2, n_hi]), n_hi=n_hi,
                    c_lo=rng.choice([0, c_hi // 3, c_hi]), c_hi=c_hi, lens=lens)
        # no more than the largest listed case, and at least one token
        if work(case)["flops"] <= 2.0e12 and sum(_lens(case)[0]):
            return case


def _lens(case):
    """(new tokens, cached positions after the append) of each sequence: the case's own."""
    r = random.Random(case["lens"])
    new, total = [], []
    for _ in range(case["batch"]):
        n = _log_int(r, case["n_lo"], case["n_hi"])
        new.append(n)
        total.append(n + r.randint(case["c_lo"], case["c_hi"]))
    return new, total


def _starts(new):
    at = [0]
    for n in new:
        at.append(at[-1] + n)
    return at


def _pair_axis(case):
    """The axis of each rotated pair: sections of a quarter for the time and equal shares of
    the rest, in turn for pairs of neighbours."""
    pairs, axes = case["rot"] // 2, case["axes"]
    if case["pairing"] == "neighbours":
        return [i % axes for i in range(pairs)]
    first = pairs if axes == 1 else pairs // 4
    rest = [1 + (i * (axes - 1)) // max(1, pairs - first) for i in range(pairs - first)]
    return [0] * first + rest


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    new, total = _lens(case)
    batch, rows, page = case["batch"], sum(new), case["page"]
    fp8 = case["kv"] == "fp8"
    dtype = torch.float8_e4m3fn if fp8 else torch.bfloat16
    k_scale, v_scale = (4.5 / 448.0, 5.0 / 448.0) if fp8 else (1.0, 1.0)

    def rand(*shape):
        return torch.randn(*shape, generator=g, device=dev).to(torch.bfloat16)

    def stored(n, scale):
        x = torch.randn(n, DIM, generator=g, device=dev)
        return (x / scale).clamp(-448.0, 448.0).to(dtype) if fp8 else x.to(dtype)

    st = dict(case=case, new=new, total=total, k_scale=k_scale, v_scale=v_scale, dtype=dtype)
    st["q"] = rand(rows, HEADS, DIM)
    st["q_start"] = torch.tensor(_starts(new), dtype=torch.int32, device=dev)
    st["seq_lens"] = torch.tensor(total, dtype=torch.int32, device=dev)
    if page:
        # pages in any order over the pool, some of them free
        per_seq = [max(1, -(-n // page)) for n in total]
        width, used = max(per_seq), sum(per_seq)
        pool = used + 3
        order = torch.randperm(pool, generator=g, device=dev).to(torch.int32)
        at = _starts(per_seq)
        table = torch.zeros(batch, width, dtype=torch.int32, device=dev)
        for b, n in enumerate(per_seq):
            table[b, :n] = order[at[b]:at[b] + n]
        st["table"] = table
        st["k"] = stored(pool * page, k_scale).view(pool, page, DIM)
        st["v"] = stored(pool * page, v_scale).view(pool, page, DIM)
    else:
        cap = max(max(total), 1)
        st["k"] = stored(batch * cap, k_scale).view(batch, cap, DIM)
        st["v"] = stored(batch * cap, v_scale).view(batch, cap, DIM)
    st["out"] = torch.empty_like(st["q"])
    if case["op"] == "append":
        kv = rand(rows, 2 * DIM)  # one projection's output, keys and values side by side
        st["new_k"], st["new_v"] = kv[:, :DIM], kv[:, DIM:]
        pairs = case["rot"] // 2
        inv = 10000.0 ** (-torch.arange(pairs, dtype=torch.float64, device=dev) / pairs)
        ang = torch.arange(MAX_POS, dtype=torch.float64, device=dev)[:, None] * inv
        st["cos_sin"] = torch.cat([ang.cos(), ang.sin()], 1).to(torch.float32)
        st["pair_axis"] = _pair_axis(case)
        st["positions"] = None  # one axis: a token's position is its cache row
        if case["axes"] > 1:
            # a grid of 18 x 31 patches a frame; the first axis counts frames
            i = torch.arange(rows, device=dev) + seed % 1000
            st["positions"] = torch.stack(
                [i // (18 * 31), i // 31 % 18, i % 31][:case["axes"]]).to(torch.int32)
            st["positions"] += 100
    if own:
        from decode_attention_10_b200 import mfa
        if page:
            st["cache"] = mfa.PagedKVCache(st["k"], st["v"], st["table"], per_seq, k_scale,
                                           v_scale)
        else:
            st["cache"] = mfa.KVCache(list(st["k"]), list(st["v"]), k_scale, v_scale)
        st["ws"] = mfa.ChunkWorkspace(batch)
        if case["op"] == "append":
            st["rope"] = mfa.Rope(st["cos_sin"], pair_axis=st["pair_axis"],
                                  interleaved=case["pairing"] == "neighbours")
    return st


def run(state):
    if state["case"]["op"] == "append":
        if own:
            from decode_attention_10_b200 import mfa
            mfa.rope_append(state["q"], state["new_k"], state["new_v"], state["cache"],
                            state["q_start"], state["seq_lens"], state["rope"],
                            positions=state["positions"], q_out=state["out"], ws=state["ws"])
            return {"q": state["out"], "k": state["k"], "v": state["v"]}
        return _append(state)
    if own:
        from decode_attention_10_b200 import mfa
        return mfa.chunk_attn(state["q"], state["cache"], state["q_start"], state["seq_lens"],
                              SCALE, out=state["out"], ws=state["ws"])
    return _attention(state)


# ------------------------------------------------------------------------ plain forms


def _rotate(x, cos, sin, pairing):
    """x [T, ..., 256] with its first 2 P dimensions rotated by angles of [T, P]."""
    p = cos.shape[1]
    cos, sin = (a.view(-1, *[1] * (x.dim() - 2), p) for a in (cos, sin))
    y = x.float()
    if pairing == "halves":
        a, b = y[..., :p], y[..., p:2 * p]
        r = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = y[..., 0:2 * p:2], y[..., 1:2 * p:2]
        r = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([r, y[..., 2 * p:]], -1)


def _append(st):
    case, q_start, seq_lens = st["case"], st["q_start"].long(), st["seq_lens"].long()
    row = torch.arange(st["q"].shape[0], device=q_start.device)
    seq = torch.searchsorted(q_start[1:], row, right=True)
    place = seq_lens[seq] - (q_start[seq + 1] - row)  # the token's cache row
    pairs = case["rot"] // 2
    pos = st["positions"].long() if st["positions"] is not None else place[None]
    axis = torch.tensor(st["pair_axis"], device=row.device)
    angle_row = pos[axis].t()
    i = torch.arange(pairs, device=row.device)
    cos, sin = st["cos_sin"][angle_row, i], st["cos_sin"][angle_row, pairs + i]
    q = _rotate(st["q"], cos, sin, case["pairing"]).to(torch.bfloat16)
    k = _rotate(st["new_k"], cos, sin, case["pairing"])
    v = st["new_v"].float()
    if case["kv"] == "fp8":
        k = (k / st["k_scale"]).clamp(-448.0, 448.0)
        v = (v / st["v_scale"]).clamp(-448.0, 448.0)
    if case["page"]:
        at = st["table"][seq, place // case["page"]].long(), place % case["page"]
    else:
        at = seq, place
    for buffer, new in ((st["k"], k), (st["v"], v)):
        # (8-bit rows are put in place as bytes)
        bits = torch.uint8 if case["kv"] == "fp8" else torch.bfloat16
        buffer.view(bits)[at] = new.to(buffer.dtype).view(bits)
    return {"q": q, "k": st["k"], "v": st["v"]}


def _softmax_attention(q, k, v, first, scale):
    """q [G, N, 64, 256] of the positions first[g] + 0 .. N - 1, k and v [G, L, 256]."""
    g, n = q.shape[:2]
    s = torch.matmul(q.reshape(g, n * HEADS, DIM), k.transpose(1, 2)).view(g, n, HEADS, -1)
    s *= scale
    hidden = (torch.arange(k.shape[1], device=q.device)
              > (first[:, None] + torch.arange(n, device=q.device))[..., None])
    s.masked_fill_(hidden[:, :, None], float("-inf"))
    s -= s.amax(-1, keepdim=True)
    s.exp_()
    total = s.sum(-1, keepdim=True)
    o = torch.matmul(s.view(g, n * HEADS, -1), v).view(g, n, HEADS, DIM)
    return o / total


def _attention(st):
    case, new, total = st["case"], st["new"], st["total"]
    q_start = _starts(new)
    n, width = max(new), max(total)

    def cached(buffer, seqs, length, scale):
        """Rows 0 .. length - 1 of some sequences, in float32."""
        if not case["page"]:
            return buffer[seqs, :length].float() * scale
        pages = st["table"][seqs, :-(-length // case["page"])].long()
        rows = buffer.view(torch.uint8)[pages].view(buffer.dtype)
        return rows.float().flatten(1, 2)[:, :length] * scale

    out = torch.empty_like(st["q"])
    if len(new) * n * HEADS * width <= SCORES and min(new) == n:
        # every sequence has the same number of new tokens: one batched product
        q = st["q"].view(len(new), n, HEADS, DIM).float()
        every = slice(None)
        k = cached(st["k"], every, width, st["k_scale"])
        v = cached(st["v"], every, width, st["v_scale"])
        first = st["seq_lens"].long() - n
        # (rows past a sequence's end are hidden from all of its tokens)
        out.copy_(_softmax_attention(q, k, v, first, SCALE).flatten(0, 1))
        return out
    for b in range(len(new)):
        if new[b]:
            one, rows = slice(b, b + 1), slice(q_start[b], q_start[b + 1])
            k = cached(st["k"], one, total[b], st["k_scale"])
            v = cached(st["v"], one, total[b], st["v_scale"])
            first = st["seq_lens"][one].long() - new[b]
            out[rows] = _softmax_attention(st["q"][rows][None].float(), k, v, first,
                                           SCALE)[0].to(out.dtype)
    return out


# ---------------------------------------------------------------- what a pass cannot avoid


def work(case):
    new, total = _lens(case)
    rows, elem = sum(new), 1 if case["kv"] == "fp8" else 2
    io = rows * HEADS * DIM * 2 * 2  # queries read, results written
    if case["op"] == "append":
        table = rows * case["rot"] * 4 + (rows * case["axes"] * 4 if case["axes"] > 1 else 0)
        return {"bytes": io + rows * 2 * DIM * (2 + elem) + table,
                "flops": rows * (HEADS + 1) * case["rot"] * 3}
    seen = sum(n * (t - n) + n * (n + 1) // 2 for n, t in zip(new, total))
    cache = sum(t for n, t in zip(new, total) if n) * 2 * DIM * elem
    return {"bytes": io + cache, "flops": seen * HEADS * DIM * 4}


# ------------------------------------------------------------------ the definition, 64 bits


def exact(case, seed):
    st = prepare(case, seed)
    return _exact_append(st) if case["op"] == "append" else _exact_attention(st)


def _exact_append(st):
    case, new, total = st["case"], st["new"], st["total"]
    table = st["cos_sin"].double()
    half = case["rot"] // 2
    if case["pairing"] == "halves":
        one, two = torch.arange(half), torch.arange(half) + half
    else:
        one, two = 2 * torch.arange(half), 2 * torch.arange(half) + 1
    where = torch.cat([torch.arange(t - n, t) for n, t in zip(new, total)]).cuda()
    owner = torch.cat([torch.full((n,), b) for b, n in enumerate(new)]).cuda()
    cos, sin = [], []
    for i in range(half):
        p = where if st["positions"] is None else st["positions"][st["pair_axis"][i]].long()
        cos.append(table[p, i])
        sin.append(table[p, half + i])
    cos, sin = torch.stack(cos, 1), torch.stack(sin, 1)

    def turned(x):
        c, s = (cos, sin) if x.dim() == 2 else (cos[:, None], sin[:, None])
        y = x.double().clone()
        a, b = x[..., one].double(), x[..., two].double()
        y[..., one] = a * c - b * s
        y[..., two] = a * s + b * c
        return y

    def kept(buffer, rows, scale):
        top = 448.0 if case["kv"] == "fp8" else float("inf")
        full = buffer.to(torch.float64)
        page, at = owner, where
        if case["page"]:
            page, at = st["table"].long()[owner, where // case["page"]], where % case["page"]
        full[page, at] = (rows / scale).clamp(-top, top)
        return full

    return {"q": turned(st["q"]), "k": kept(st["k"], turned(st["new_k"]), st["k_scale"]),
            "v": kept(st["v"], st["new_v"].double(), st["v_scale"])}


def _exact_attention(st):
    case, new, total = st["case"], st["new"], st["total"]
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device=st["q"].device)
    row = 0
    for b, (n, t) in enumerate(zip(new, total)):
        if n == 0:
            continue
        if case["page"]:
            ids = st["table"][b].tolist()[:-(-t // case["page"])]
            k = torch.cat([st["k"][i] for i in ids]).double()[:t] * st["k_scale"]
            v = torch.cat([st["v"][i] for i in ids]).double()[:t] * st["v_scale"]
        else:
            k = st["k"][b][:t].double() * st["k_scale"]
            v = st["v"][b][:t].double() * st["v_scale"]
        step = max(1, (1 << 28) // (HEADS * t))  # tokens at a time
        for lo in range(0, n, step):
            hi = min(n, lo + step)
            seen = t - n + hi  # positions that the last of these tokens sees
            x = st["q"][row + lo:row + hi].double()
            s = torch.einsum("nhd,ld->nhl", x, k[:seen]) * SCALE
            for i in range(lo, hi):
                s[i - lo, :, t - n + i + 1:] = -math.inf
            out[row + lo:row + hi] = torch.einsum("nhl,ld->nhd", torch.softmax(s, -1),
                                                  v[:seen])
        row += n
    return out
