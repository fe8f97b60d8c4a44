"""The attention of a chunk of new tokens (mfa_chunk_attn) against its plain form in 64 bits,
at the lengths, layouts and masks where it can go wrong."""

import pytest
import torch

from chunk_util import DIM, HEADS, Batch, check

pytestmark = pytest.mark.gpu

KV = pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
LAYOUT = pytest.mark.parametrize("page", [0, 64, 128, 512], ids=["buffers", "p64", "p128", "p512"])


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from decode_attention_10_b200 import build, mfa
    build.build()
    mfa.load()


def run(b, ws=None, **kw):
    from decode_attention_10_b200 import mfa
    ws = ws or mfa.ChunkWorkspace(b.batch)
    cache = b.cache()
    out = mfa.chunk_attn(b.q, cache, b.q_start, b.seq_lens, ws=ws, **kw)
    assert mfa.get_error(ws) == 0
    return out


@KV
@LAYOUT
@pytest.mark.parametrize("new,cached", [
    ([1], [0]), ([1], [1]), ([2], [0]), ([3], [126]), ([4], [124]), ([4], [125]), ([5], [127]),
    ([1], [127]), ([1], [128]), ([7], [60]), ([130], [0]), ([67], [301]), ([9], [2000]),
])
def test_one_sequence(fp8, page, new, cached):
    b = Batch(new, cached, fp8, page, seed=sum(new) + sum(cached))
    check(run(b), b)


@KV
@LAYOUT
def test_ragged_batch_with_empty_sequences(fp8, page):
    # decoding sequences, chunks of every remainder of 4, and sequences with no new token
    new = [1, 0, 4, 33, 1, 0, 2, 65, 3, 1, 0]
    cached = [500, 70, 128, 95, 0, 0, 1023, 7, 62, 129, 300]
    b = Batch(new, cached, fp8, page, seed=3, spare=40)
    check(run(b), b)


@KV
def test_long_context_is_split_and_joined(fp8):
    b = Batch([3, 1], [20001, 9000], fp8, 64, seed=4)
    check(run(b), b)


@KV
def test_chunk_over_a_long_context(fp8):
    b = Batch([150], [5003], fp8, 128, seed=5)
    check(run(b), b)


@KV
def test_many_sequences(fp8):
    new = [(7 * i) % 5 for i in range(1024)]
    cached = [(37 * i) % 300 for i in range(1024)]
    b = Batch(new, cached, fp8, 64, seed=6)
    check(run(b), b)


@KV
@LAYOUT
def test_rows_past_the_end_are_never_weighted(fp8, page):
    # NaN (and, in bf16, infinities) past every sequence's end, in its own pages and rows
    for tail in (float("nan"),) if fp8 else (float("nan"), float("inf")):
        b = Batch([5, 1, 4, 66], [123, 64, 0, 190], fp8, page, seed=7, spare=70, tail=tail)
        out = run(b)
        assert torch.isfinite(out).all()
        check(out, b)


@KV
@LAYOUT
@pytest.mark.parametrize("cached", [0, 61, 125, 126, 127, 200])
def test_a_token_s_bad_rows_reach_it_and_later_tokens_only(fp8, page, cached):
    # the K and V rows of new token 2 (of 7) hold NaN; the V row of token 5 an infinity
    b = Batch([7], [cached], fp8, page, seed=8, spare=10)
    clean = run(b)
    nan = 0x7F if fp8 else 0x7FC0
    for which in ("k", "v"):
        set_row(b, which, 0, cached + 2, nan)
    if not fp8:
        set_row(b, "v", 0, cached + 5, 0x7F80)
    out = run(b)
    assert torch.equal(out[:2], clean[:2])
    assert out[2:].isnan().all()
    b = Batch([7], [cached], fp8, page, seed=8, spare=10)
    set_row(b, "v", 0, cached + 5, nan, dims=slice(3, 4))  # one value of one row
    out = run(b)
    assert torch.equal(out[:5], clean[:5])
    assert out[5:, :, 3].isnan().all()
    out[5:, :, 3] = clean[5:, :, 3]  # its other values weigh as ever
    check(out, Batch([7], [cached], fp8, page, seed=8, spare=10))


def set_row(b, which, seq, row, bits, dims=slice(0, DIM)):
    buf = b.k if which == "k" else b.v
    t = buf if b.page else buf[seq]
    raw = t.view(torch.uint8 if b.fp8 else torch.int16)
    if b.page:
        raw[int(b.table[seq, row // b.page]), row % b.page, dims] = bits
    else:
        raw[row, dims] = bits


@KV
def test_a_bad_query_reaches_its_own_row_only(fp8):
    b = Batch([6], [100], fp8, 64, seed=9)
    clean = run(b)
    b.q[2, 17] = float("nan")
    b.q[4, 3, 5] = float("inf")
    out = run(b)
    keep = torch.ones(6, HEADS, dtype=torch.bool)
    keep[2, 17] = keep[4, 3] = False
    assert torch.equal(out[keep], clean[keep])
    assert out[2, 17].isnan().all()


def test_scores_of_minus_infinity():
    # keys of -inf in visible rows: weight zero next to finite ones, NaN where all are so
    b = Batch([4], [300], False, 64, seed=10)
    b.q.fill_(0.5)
    for row in range(0, 256):
        set_row(b, "k", 0, row, 0xFF80 - 0x10000)
    out = run(b)
    k, v = b.values("k", 0), b.values("v", 0)
    for i in range(4):
        s = (b.q[i].double() @ k[256:301 + i].T) / 16
        want = torch.softmax(s, -1) @ v[256:301 + i]
        mag = torch.softmax(s, -1) @ v[256:301 + i].abs()
        assert ((out[i].double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -7 * mag).all()
    b = Batch([4], [3], False, 64, seed=10)
    b.q.fill_(0.5)
    for row in range(0, 5):
        set_row(b, "k", 0, row, 0xFF80 - 0x10000)
    out = run(b)
    assert out[:2].isnan().all() and torch.isfinite(out[2:]).all()


@KV
@pytest.mark.parametrize("q_scale", [0.01, 8.0, 40.0])
def test_flat_and_sharp_softmax(fp8, q_scale):
    b = Batch([9, 70], [700, 450], fp8, 128, seed=11, q_scale=q_scale)
    check(run(b), b)


@KV
def test_rising_scores_rescale_at_every_block(fp8):
    # keys grow along the context, so every block raises the running maximum
    b = Batch([5], [1200], fp8, 0, seed=12)
    grow = torch.linspace(0.02, 1.0, b.total[0], device="cuda")[:, None]
    u = torch.randn(DIM, generator=torch.Generator().manual_seed(1)).cuda()
    rows = grow * u
    b.k[0][:] = (rows / b.k_scale).clamp(-448, 448).to(b.k[0].dtype)
    b.q[:] = (u + 0.1 * b.q.float()).to(torch.bfloat16)
    check(run(b), b)


@KV
def test_rows_of_no_sequence_stay(fp8):
    b = Batch([3, 6], [40, 200], fp8, 64, seed=13, lead=2, behind=9)
    out = torch.full_like(b.q, 77.0)
    run(b, out=out)
    check(out, b)
    assert (out[:2] == 77.0).all() and (out[b.starts[-1]:] == 77.0).all()


@KV
def test_scale_is_an_argument(fp8):
    b = Batch([5], [333], fp8, 64, seed=14)
    check(run(b, scale=0.17), b, scale=0.17)


@KV
@pytest.mark.parametrize("scale,q_scale", [(1e-37, 1e-5), (1e-20, 1e-30), (3e-6, 1.0), (50.0, 1e-4)])
def test_tiny_and_large_scales(fp8, scale, q_scale):
    # down to factors of the scores that float32 cannot hold
    b = Batch([6], [250], fp8, 64, seed=27, q_scale=q_scale)
    check(run(b, scale=scale), b, scale=scale)


@KV
def test_agrees_with_the_decode_attention(fp8):
    # one new token a sequence is mfa_decode_attn
    from decode_attention_10_b200 import mfa
    b = Batch([1] * 9, [0, 5, 127, 128, 129, 700, 2047, 64, 63], fp8, 128, seed=15)
    out = run(b)
    ws = mfa.Workspace(b.batch)
    ref = mfa.decode_attn(b.q, b.cache(), b.seq_lens, ws=ws)
    check(out, b)
    check(ref, b)
    assert (out.float() - ref.float()).abs().max() <= 2e-2


@KV
def test_same_call_same_bits(fp8):
    b = Batch([70, 1, 5, 1], [3000, 9000, 100, 0], fp8, 64, seed=16)
    first = run(b)
    for _ in range(3):
        assert torch.equal(run(b), first)


def test_errors_are_reported_and_zero_filled():
    from decode_attention_10_b200 import mfa
    b = Batch([2, 3, 4, 2], [50, 60, 0, 200], False, 64, seed=17)
    ws = mfa.ChunkWorkspace(4)
    cache = b.cache()
    good = run(b)
    bad = b.seq_lens.clone()
    bad[1] = 129  # over the capacity of two pages
    out = torch.full_like(b.q, 5.0)
    mfa.chunk_attn(b.q, cache, b.q_start, bad, out=out, ws=ws)
    assert mfa.get_error(ws) == 3 and mfa.get_error(ws) == 0
    assert (out[2:5] == 0).all()
    assert torch.equal(out[:2], good[:2]) and torch.equal(out[5:], good[5:])
    for length in (3, 0, -7):  # fewer positions than new tokens
        bad = b.seq_lens.clone()
        bad[2] = length
        out = torch.full_like(b.q, 5.0)
        mfa.chunk_attn(b.q, cache, b.q_start, bad, out=out, ws=ws)
        assert mfa.get_error(ws) == 6
        assert (out[5:9] == 0).all()
        assert torch.equal(out[:5], good[:5]) and torch.equal(out[9:], good[9:])
    # ranges that do not hold together: nothing is computed
    for starts in ([0, 2, 5, 9, 40], [-3, 2, 5, 9, 11], [0, 2, 1, 4, 11], [0, 2, 5, 900, 11]):
        out = torch.full_like(b.q, 5.0)
        q_start = torch.tensor(starts, dtype=torch.int32, device="cuda")
        mfa.chunk_attn(b.q, cache, q_start, b.seq_lens, out=out, ws=ws)
        assert mfa.get_error(ws) == 1 and (out == 5.0).all()
    out = torch.full_like(b.q, 5.0)
    mfa.chunk_attn(b.q, cache, b.q_start, b.seq_lens, out=out, ws=ws)
    assert mfa.get_error(ws) == 0 and torch.equal(out, good)


def test_table_without_chunk_maps_is_refused():
    from decode_attention_10_b200 import mfa
    import ctypes
    b = Batch([2], [50], False, 0, seed=18)
    lib = mfa.load()
    small = lib.mfa_kv_table_bytes(1)
    table = torch.zeros(small + 512, dtype=torch.uint8, device="cuda")
    arr = (ctypes.c_void_p * 1)(b.k[0].data_ptr())
    arv = (ctypes.c_void_p * 1)(b.v[0].data_ptr())
    cap = (ctypes.c_int32 * 1)(b.cap[0])
    assert lib.mfa_kv_table_init(table.data_ptr(), small, 1, 0, arr, arv, cap, None) == 0
    assert (table[small:] == 0).all()
    cache = b.cache()
    cache.desc.table = table.data_ptr()
    ws = mfa.ChunkWorkspace(1)
    out = torch.full_like(b.q, 5.0)
    mfa.chunk_attn(b.q, cache, b.q_start, b.seq_lens, out=out, ws=ws)
    assert mfa.get_error(ws) == 1 and (out == 5.0).all()
    # a stated layout that the table contradicts
    cache = b.cache()
    cache.desc.page_size = 64
    mfa.chunk_attn(b.q, cache, b.q_start, b.seq_lens, out=out, ws=ws)
    assert mfa.get_error(ws) == 1 and (out == 5.0).all()


@KV
@LAYOUT
def test_fewer_sequences_than_the_table(fp8, page):
    # a description of a table's first sequences
    from decode_attention_10_b200 import mfa
    b = Batch([3, 9, 1, 5], [60, 200, 70, 1], fp8, page, seed=23)
    cache = b.cache()
    cache.desc.batch = cache.batch = 2
    ws = mfa.ChunkWorkspace(2)
    out = mfa.chunk_attn(b.q[:12], cache, b.q_start[:3], b.seq_lens[:2], ws=ws)
    ref, tol = b.reference()
    assert mfa.get_error(ws) == 0
    assert ((out.double() - ref[:12]).abs() <= tol[:12]).all()


def test_page_outside_the_pool_reads_as_zeros():
    # as in mfa_decode_attn: such a page's keys and values are zeros
    b = Batch([3], [300], False, 64, seed=19)
    ref = run(b)
    b.table[0, 1] = 10 ** 6
    out = run(b)
    assert torch.isfinite(out).all() and not torch.equal(out, ref)
    b.table[0, 1] = -1
    assert torch.equal(run(b), out)


@KV
def test_captured_and_replayed(fp8):
    # replays read the lengths, starts and pages of their time
    from decode_attention_10_b200 import mfa
    a = Batch([4, 1, 20], [100, 700, 0], fp8, 64, seed=20, spare=500)
    ws = mfa.ChunkWorkspace(3)
    cache = a.cache()
    out = torch.zeros_like(a.q)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        mfa.chunk_attn(a.q, cache, a.q_start, a.seq_lens, out=out, ws=ws)
    torch.cuda.synchronize()
    want = out.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        mfa.chunk_attn(a.q, cache, a.q_start, a.seq_lens, out=out, ws=ws)
        mfa.chunk_attn(a.q, cache, a.q_start, a.seq_lens, out=out, ws=ws)
    out.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    a.q_start.copy_(torch.tensor([0, 1, 5, 25], dtype=torch.int32))
    a.seq_lens.copy_(torch.tensor([101, 704, 20], dtype=torch.int32))
    a.q.copy_(torch.randn_like(a.q.float()).to(torch.bfloat16))
    fresh = mfa.chunk_attn(a.q, cache, a.q_start, a.seq_lens)
    out.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, fresh) and mfa.get_error(ws) == 0


def test_two_calls_on_two_streams_with_workspaces_of_their_own():
    from decode_attention_10_b200 import mfa
    bs = [Batch([50, 3], [2000, 4000], False, 64, seed=21), Batch([7], [6000], True, 0, seed=22)]
    caches = [b.cache() for b in bs]
    wss = [mfa.ChunkWorkspace(b.batch) for b in bs]
    want = [run(b) for b in bs]
    streams = [torch.cuda.Stream() for _ in bs]
    outs = [torch.zeros_like(b.q) for b in bs]
    torch.cuda.synchronize()
    for _ in range(5):
        for b, c, w, s, o in zip(bs, caches, wss, streams, outs):
            mfa.chunk_attn(b.q, c, b.q_start, b.seq_lens, out=o, ws=w, stream=s)
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert torch.equal(o, w)


def test_own_results_and_workspace_on_a_given_stream():
    # what a call allocates itself is not handed out again before the given stream is done
    from decode_attention_10_b200 import mfa
    b = Batch([300, 2], [6000, 9000], False, 64, seed=23)
    cache, want, s = b.cache(), run(b), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(6):
        out = mfa.chunk_attn(b.q, cache, b.q_start, b.seq_lens, stream=s)
        junk = [torch.full((1 << 23,), float("nan"), device="cuda") for _ in range(3)]
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        del junk


@KV
@pytest.mark.parametrize("new,cached", [
    ([1], [60000]), ([12], [9000]), ([13], [9000]), ([2, 0, 3, 7], [30000, 5, 257, 8000]),
    ([1] * 12, [3000 + 700 * i for i in range(12)]),
    ([1] * 13, [3000 + 700 * i for i in range(13)]),
    ([1] * 6, [9000] * 6), ([1] * 7, [9000] * 7), ([64], [3000]), ([65], [3000]),
    ([25, 0, 39], [700, 64, 5000]), ([1] * 64, [900] * 64), ([1] * 65, [900] * 65),
])
def test_few_tokens_over_long_contexts(fp8, new, cached):
    # many parts a tile, on both sides of the merge's choices (6 tiles, 64 tokens)
    b = Batch(new, cached, fp8, 256, seed=24)
    check(run(b), b)


def test_memory_of_another_device_is_refused():
    from decode_attention_10_b200 import mfa
    b = Batch([3], [40], False, 64, seed=25)
    cache, ws = b.cache(), mfa.ChunkWorkspace(1)
    cache.device_index = ws.device_index = torch.cuda.current_device() + 1
    with pytest.raises(ValueError, match="not on the current device"):
        mfa.chunk_attn(b.q, cache, b.q_start, b.seq_lens, ws=ws)
    k = torch.zeros(3, DIM, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError, match="not on the current device"):
        mfa.rope_append(None, k, k, cache, b.q_start, b.seq_lens, ws=ws)


def test_results_over_the_queries_are_refused():
    from decode_attention_10_b200 import mfa
    b = Batch([5], [40], False, 64, seed=26)
    with pytest.raises(mfa.MfaError, match="INVALID_ARG"):
        mfa.chunk_attn(b.q, b.cache(), b.q_start, b.seq_lens, out=b.q)


@KV
@pytest.mark.parametrize("new", [1, 301], ids=["parts", "tiles"])
@pytest.mark.parametrize("keys,score", [(8192, 10), (32768, 11), (65536, 12), (65536, 14)])
def test_a_dominating_key_leaves_the_others_their_weight(fp8, new, keys, score):
    # The first key has half to nine tenths of every row's weight and a value of zero; the rest of the
    # weight is spread over thousands of keys with values around 1.
    b = Batch([new], [keys - new], fp8, 0, seed=28)
    if fp8:
        b.k_scale, b.v_scale = 1.0, 1.0 / 16
    g = torch.Generator().manual_seed(29)
    k = torch.randn(keys, DIM, generator=g)
    k[:, 0], k[0] = 0.0, 0.0
    k[0, 0] = 16.0 * score  # q . k / 16, with a 1 in q
    v = 1.0 + 0.5 * torch.randn(keys, DIM, generator=g)
    v[0] = 0.0
    b.k[0].copy_(k / b.k_scale)
    b.v[0].copy_(v / b.v_scale)
    b.q[:, :, 0] = 1.0
    out = run(b).double()
    kd, vd = b.values("k", 0), b.values("v", 0)
    for t in sorted({0, 3, new // 2, new - 1} & set(range(new))):
        end = keys - new + t + 1
        q = b.q[t].double()
        s = q @ kd[:end].T / 16
        p = torch.softmax(s, -1)
        want = p @ vd[:end]
        top = p.amax(-1, keepdim=True)
        assert (top > 0.4).all() and (want > 0.05).all()
        # Each weight's rounding to bf16: half a step, 2^-8 of it. FP8: a weight of w = 2^8 p / top
        # or more is an f16 (2^-11) and then e4m3 + e5m2: from 2^-6 up within 2^-8 of its power of
        # two; below, the e5m2 part is at most 2^-10, off by 2^-14 at most, and by 2^-3 of itself or
        # half of the smallest step, 2^-17.
        one = (2.0 ** -8 + 2.0 ** -11) * p
        if fp8:
            one = one + torch.minimum(2.0 ** -22 * top, 2.0 ** -3 * p + 2.0 ** -25 * top)
        # These errors have either sign: within 8 standard deviations of their sum, a step's error
        # taken as its largest, and a mean of at most 2^-6 of the weights' sum (steps of up to a
        # quarter of a weight, (1/4)^2 / 12 times the few that a density falls by over a weight).
        off = 8 * (one ** 2 @ vd[:end] ** 2).sqrt() + (2.0 ** -6 if fp8 else 0) * (p @ vd[:end].abs())
        # the scores' float32 sums, and FP8 q as a pair (chunk_util); the result's rounding
        dot = (q.abs() @ kd[:end].abs().T).amax(-1, keepdim=True) / 16
        err = 256 * 2.0 ** -23 * dot
        if fp8:
            err = err + 2.0 ** -17 * q.abs().amax(-1, keepdim=True) * kd.abs().sum(-1).max() / 16
        tol = 2.0 ** -8 * want.abs() + off + 2 * err * (p @ vd[:end].abs() + want.abs())
        d = (out[t] - want).abs()
        assert (d <= tol).all(), (t, float(d.max()), float(tol.min()), float((d / want).max()))


@KV
@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("new,cached", [(1, 0), (1, 129), (6, 100), (6, 9000), (66, 3)])
def test_a_query_with_an_infinity_is_nan(fp8, new, cached, bad):
    # inf times any key is an infinity or NaN, so the row has no softmax
    b = Batch([new], [cached], fp8, 64, seed=30)
    clean = run(b)
    t = new // 2
    b.q[t, 3, 5] = b.q[new - 1, 63, 255] = bad
    out = run(b)
    keep = torch.ones(new, HEADS, dtype=torch.bool)
    keep[t, 3] = keep[new - 1, 63] = False
    assert out[t, 3].isnan().all() and out[new - 1, 63].isnan().all()
    assert torch.equal(out[keep], clean[keep])


@KV
@pytest.mark.parametrize("rise", [0.3, 1.5, 2.5, 2.7, 2.8, 4.0, 5.4, 5.6])
def test_scores_above_the_running_maximum(fp8, rise):
    # later keys score up to `rise` above the first block's, below and above what raises the running
    # maximum (4 in log2, 2.77, for FP8; 8, 5.55, for bf16): weights of up to 2^12, or 2^8
    b = Batch([1, 6], [1500, 1500], fp8, 0, seed=31)
    b.k_scale = 1.0 / 64 if fp8 else 1.0
    g = torch.Generator().manual_seed(32)
    for i in range(2):
        up = torch.rand(b.total[i], generator=g) * rise
        up[:128], up[700] = 0.0, rise
        k = 0.05 * torch.randn(b.total[i], DIM, generator=g)
        k[:, 0] = up
        b.k[i].copy_((k / b.k_scale).clamp(-448, 448))
    b.q[:, :, 0] = 16.0
    check(run(b), b)
