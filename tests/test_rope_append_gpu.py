"""The rotated append (mfa_rope_append) against its plain form in 64 bits, and the run of a
prompt and its decoding through the operators together."""

import pytest
import torch

from chunk_util import DIM, F64, Batch, angles, rotate

pytestmark = pytest.mark.gpu

KV = pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from decode_attention_10_b200 import build, mfa
    build.build()
    mfa.load()


def new_rows(rows, seed, ld=2 * DIM):
    g = torch.Generator().manual_seed(1000 + seed)
    kv = torch.randn(max(1, rows), ld, generator=g).to(torch.bfloat16).cuda()
    return kv[:, :DIM], kv[:, ld - DIM:]


def make_rope(rot=256, axes=1, interleaved=False, max_pos=4096):
    from decode_attention_10_b200 import mfa
    p = rot // 2
    pair_axis = [min(axes - 1, (i * axes) // p) for i in range(p)] if not interleaved \
        else [i % axes for i in range(p)]
    return mfa.Rope(mfa.rope_table(max_pos, rot), pair_axis, interleaved), pair_axis


def snapshot(b):
    bufs = [b.k, b.v] if b.page else [*b.k, *b.v]
    return [t.view(torch.uint8).clone() for t in bufs]


def expected(b, k, v, rope, pair_axis, positions):
    """(rotated q, rotated k, v) in float64 and the magnitude that bounds their arithmetic."""
    place = torch.cat([torch.arange(t - n, t) for n, t in zip(b.new, b.total)]).cuda()
    sl = slice(b.starts[0], b.starts[-1])
    pos = place[None] if positions is None else positions[:, sl]
    c, s = angles(rope.table, rope.rot_dim, pair_axis, pos)
    q, k, v = b.q[sl].to(F64), k[sl].to(F64), v[sl].to(F64)
    inter = bool(rope.desc.interleaved)
    mag = [rotate(x.abs(), c.abs(), -s.abs(), inter).abs()
           + rotate(x.abs(), c.abs(), s.abs(), inter).abs() for x in (q, k)]
    return rotate(q, c, s, inter), rotate(k, c, s, inter), v, mag


def verify(b, before, q_out, k, v, rope, pair_axis, positions):
    q_ref, k_ref, v_ref, (q_mag, k_mag) = expected(b, k, v, rope, pair_axis, positions)
    sl = slice(b.starts[0], b.starts[-1])
    # half a bf16 step of the result, and three float32 roundings of its two products
    tol = 2.0 ** -8 * q_ref.abs() + 2.0 ** -22 * q_mag
    assert ((q_out[sl].to(F64) - q_ref).abs() <= tol).all()
    at = 0
    for i in range(b.batch):
        n, t = b.new[i], b.total[i]
        for which, ref, mag, scale in (("k", k_ref, k_mag, b.k_scale),
                                       ("v", v_ref, v_ref.abs(), b.v_scale)):
            got = b.stored(which, i)[t - n:].to(F64)
            want = ref[at:at + n] / scale
            if b.fp8:
                want = want.clamp(-448, 448)
                # half an e4m3 step: 2^-4 of a normal value, 2^-10 below
                tol = (2.0 ** -4 * want.abs()).clamp_min(2.0 ** -10)
            else:
                tol = 2.0 ** -8 * want.abs()
            tol = tol + 2.0 ** -21 * mag[at:at + n] / scale
            assert ((got - want).abs() <= tol).all(), (i, which)
        at += n
    # every other byte of the cache as it was: put the old rows back and compare
    olds = iter(before)
    for which in ("k", "v"):
        if b.page:
            old, now = next(olds), (b.k if which == "k" else b.v).view(torch.uint8).clone()
            for i in range(b.batch):
                for r in range(b.total[i] - b.new[i], b.total[i]):
                    page = int(b.table[i, r // b.page])
                    now[page, r % b.page] = old[page, r % b.page]
            assert torch.equal(now, old)
        else:
            for i in range(b.batch):
                old = next(olds)
                now = (b.k if which == "k" else b.v)[i].view(torch.uint8).clone()
                now[b.total[i] - b.new[i]:b.total[i]] = old[b.total[i] - b.new[i]:b.total[i]]
                assert torch.equal(now, old)


@KV
@pytest.mark.parametrize("page", [0, 64, 256], ids=["buffers", "p64", "p256"])
@pytest.mark.parametrize("rot,axes,interleaved", [(256, 1, False), (256, 3, True), (64, 2, False),
                                                  (208, 4, True), (16, 1, True), (96, 3, False)])
def test_rotated_append(fp8, page, rot, axes, interleaved):
    from decode_attention_10_b200 import mfa
    b = Batch([1, 0, 70, 3, 1], [64, 9, 100, 0, 255], fp8, page, seed=rot + axes, spare=3)
    rope, pair_axis = make_rope(rot, axes, interleaved)
    k, v = new_rows(b.rows, rot)
    positions = None
    if axes > 1:
        positions = torch.randint(0, 4096, (axes, b.rows), dtype=torch.int32, device="cuda",
                                  generator=torch.Generator("cuda").manual_seed(2))
        positions[:, 0], positions[:, 1] = 0, 4095
    before = snapshot(b)
    ws = mfa.Workspace(b.batch)
    q_out = mfa.rope_append(b.q, k, v, b.cache(), b.q_start, b.seq_lens, rope, positions, ws=ws)
    assert mfa.get_error(ws) == 0
    verify(b, before, q_out, k, v, rope, pair_axis, positions)


def test_given_positions_equal_to_the_rows_change_nothing():
    from decode_attention_10_b200 import mfa
    b = Batch([5, 2], [30, 200], False, 64, seed=1)
    rope, _ = make_rope()
    k, v = new_rows(b.rows, 1)
    first = mfa.rope_append(b.q, k, v, b.cache(), b.q_start, b.seq_lens, rope)
    pos = torch.tensor([30, 31, 32, 33, 34, 200, 201], dtype=torch.int32, device="cuda")
    again = mfa.rope_append(b.q, k, v, b.cache(), b.q_start, b.seq_lens, rope, pos)
    assert torch.equal(first, again)


@KV
def test_in_place_and_append_only(fp8):
    from decode_attention_10_b200 import mfa
    for rot in (256, 128):
        b = Batch([5, 2], [30, 200], fp8, 64, seed=rot)
        rope, _ = make_rope(rot)
        k, v = new_rows(b.rows, 2)
        want = mfa.rope_append(b.q, k, v, b.cache(), b.q_start, b.seq_lens, rope)
        after = snapshot(b)
        q = b.q.clone()
        assert mfa.rope_append(q, k, v, b.cache(), b.q_start, b.seq_lens, rope,
                               q_out=q) is q
        assert torch.equal(q, want)
        assert mfa.rope_append(None, k, v, b.cache(), b.q_start, b.seq_lens, rope) is None
        for x, y in zip(snapshot(b), after):
            assert torch.equal(x, y)


@KV
def test_append_without_rotation(fp8):
    from decode_attention_10_b200 import mfa
    b = Batch([3, 66], [61, 0], fp8, 64, seed=5)
    k, v = new_rows(b.rows, 5, ld=520)
    mfa.rope_append(None, k, v, b.cache(), b.q_start, b.seq_lens)
    for i in range(2):
        rows = slice(b.starts[i], b.starts[i + 1])
        for which, src, s in (("k", k, b.k_scale), ("v", v, b.v_scale)):
            got = b.stored(which, i)[b.cached[i]:]
            if fp8:
                want = (src[rows].float() / s).clamp(-448, 448).to(torch.float8_e4m3fn)
                assert torch.equal(got.view(torch.uint8), want.view(torch.uint8))
            else:
                assert torch.equal(got, src[rows])


def test_rows_of_no_sequence_and_other_rows_stay():
    from decode_attention_10_b200 import mfa
    b = Batch([2, 3], [10, 70], False, 64, seed=6, lead=1, behind=4)
    rope, pair_axis = make_rope()
    k, v = new_rows(b.rows, 6)
    before = snapshot(b)
    q_out = torch.full_like(b.q, 9.0)
    mfa.rope_append(b.q, k, v, b.cache(), b.q_start, b.seq_lens, rope, q_out=q_out)
    verify(b, before, q_out, k, v, rope, pair_axis, None)
    assert (q_out[:1] == 9.0).all() and (q_out[b.starts[-1]:] == 9.0).all()


def test_bad_rows_positions_and_pages_write_nothing():
    from decode_attention_10_b200 import mfa
    b = Batch([2, 3], [62, 60], False, 64, seed=7)
    rope, _ = make_rope(max_pos=100)
    k, v = new_rows(b.rows, 7)
    cache, ws = b.cache(), mfa.Workspace(2)

    def call(lens=None, positions=None, starts=None):
        q_out = torch.full_like(b.q, 9.0)
        mfa.rope_append(b.q, k, v, cache, starts if starts is not None else b.q_start,
                        lens if lens is not None else b.seq_lens, rope, positions, q_out=q_out,
                        ws=ws)
        return q_out, mfa.get_error(ws)

    assert call()[1] == 0
    # the second sequence ends one past its 64 rows: its last token has no row
    out, err = call(lens=torch.tensor([64, 65], dtype=torch.int32, device="cuda"))
    assert err == 3 and (out[4] == 9.0).all() and (out[:4] != 9.0).any()
    for lens in ([64, 1], [64, -5]):
        out, err = call(lens=torch.tensor(lens, dtype=torch.int32, device="cuda"))
        assert err == 3 and (out[2] == 9.0).all()
    # positions outside the table
    for p in (-1, 100, 2 ** 31 - 1):
        pos = torch.tensor([3, p, 5, 6, 7], dtype=torch.int32, device="cuda")
        out, err = call(positions=pos)
        assert err == 3 and (out[1] == 9.0).all() and not (out[0] == 9.0).all()
    # a page outside the pool
    old = b.table.clone()
    b.table[0, 0] = 10 ** 6
    before = snapshot(b)
    out, err = call()
    assert err == 3 and (out[:2] == 9.0).all()
    b.table.copy_(old)
    used = set(b.table[1, :1].tolist())
    for x, y in zip(snapshot(b), before):
        for page in range(x.shape[0]):
            if page not in used:
                assert torch.equal(x[page], y[page])


def test_many_sequences_and_max_batch():
    from decode_attention_10_b200 import mfa
    new = [(3 * i) % 4 for i in range(1024)]
    cached = [(5 * i) % 60 for i in range(1024)]
    b = Batch(new, cached, False, 64, seed=8)
    rope, pair_axis = make_rope()
    k, v = new_rows(b.rows, 8)
    before = snapshot(b)
    q_out = mfa.rope_append(b.q, k, v, b.cache(), b.q_start, b.seq_lens, rope)
    verify(b, before, q_out, k, v, rope, pair_axis, None)


def test_far_positions_turn_by_the_right_angle():
    # position 65535: an angle formed in float32 would be off by up to 2^-9 radians
    from decode_attention_10_b200 import mfa
    t = mfa.rope_table(65536, 256)
    i = torch.arange(128, dtype=torch.float64)
    want = 65535.0 * 10000.0 ** (-2.0 * i / 256)
    assert (t[65535, :128].cpu().double() - want.cos()).abs().max() <= 2.0 ** -24
    assert (t[65535, 128:].cpu().double() - want.sin()).abs().max() <= 2.0 ** -24


@KV
@pytest.mark.parametrize("page", [0, 64])
def test_prompt_in_chunks_then_decoding(fp8, page):
    """A batch's prompts in ragged chunks, then decoded tokens: every step projects its
    queries with the library, rotates and appends, and attends; the results are those of the
    plain form over the whole sequence at once."""
    from decode_attention_10_b200 import mfa
    from decode_attention_10_b200 import workloads as W
    total = [150, 37, 260]
    b = Batch([0, 0, 0], total, fp8, page, seed=9, tail=float("nan"), spare=4)
    for buf in ([b.k, b.v] if page else [*b.k, *b.v]):
        buf.view(torch.uint8).fill_(0x7F)  # nothing cached yet: rows of NaN
    inp = W.generate([1], W.KV_BF16, seed=3)
    w_qdown, gamma, w_qup = inp.w_qdown.cuda(), inp.gamma.cuda(), inp.w_qup.cuda()
    w_kv = torch.cat([inp.w_k, inp.w_v], 1).cuda()
    g = torch.Generator().manual_seed(4)
    x = [torch.randn(t, 7168, generator=g).to(torch.bfloat16).cuda() for t in total]
    rope, pair_axis = make_rope(256, 1, False, 512)
    cache, ws = b.cache(), mfa.ChunkWorkspace(3)
    done, outs, qs, ks, vs = [0] * 3, [[], [], []], [[], [], []], [[], [], []], [[], [], []]
    steps = [[100, 30, 1], [0, 5, 200], [46, 1, 55], [1, 1, 1], [1, 0, 1], [1, 0, 1], [1, 0, 1]]
    for step, new in enumerate(steps):
        xs = torch.cat([x[i][done[i]:done[i] + new[i]] for i in range(3)])
        starts = torch.tensor([0, new[0], new[0] + new[1], sum(new)], dtype=torch.int32).cuda()
        lens = torch.tensor([d + n for d, n in zip(done, new)], dtype=torch.int32).cuda()
        pws = mfa.Workspace(xs.shape[0])
        q = mfa.query_proj(xs, w_qdown, gamma, w_qup, ws=pws)
        kv = (xs.float() @ w_kv.float()).to(torch.bfloat16)
        q_raw = q.clone()
        mfa.rope_append(q, kv[:, :DIM], kv[:, DIM:], cache, starts, lens, rope, q_out=q, ws=ws)
        if step == 3:  # all sequences decode one token: the decode attention serves too
            o = mfa.decode_attn(q, cache, lens, ws=ws)
        else:
            o = mfa.chunk_attn(q, cache, starts, lens, ws=ws)
        at = 0
        for i in range(3):
            rows = slice(at, at + new[i])
            at += new[i]
            outs[i].append(o[rows])
            qs[i].append(q_raw[rows])
            ks[i].append(kv[rows, :DIM])
            vs[i].append(kv[rows, DIM:])
            done[i] += new[i]
    assert mfa.get_error(ws) == 0 and done == total
    # the same in one piece: the stored rows are the rotated rows, rounded; the results those
    # of the rotated, rounded queries over the stored rows
    for i in range(3):
        q, k, v, o = (torch.cat(t[i]) for t in (qs, ks, vs, outs))
        c, s = angles(rope.table, 256, pair_axis, torch.arange(total[i], device="cuda")[None])
        k_ref = rotate(k.to(F64), c, s, False) / b.k_scale
        got = b.stored("k", i).to(F64)
        step8 = (2.0 ** -4 * k_ref.abs()).clamp_min(2.0 ** -10) if fp8 else 2.0 ** -8 * k_ref.abs()
        lim = step8 + 2.0 ** -20 * k_ref.abs().max()
        assert ((got - k_ref).abs() <= lim).all()
        one = Batch([total[i]], [0], fp8, page, seed=1)
        one.q = rotate(q.to(F64), c, s, False).to(torch.bfloat16)
        one.values = lambda which, _, i=i: b.values(which, i)
        ref, tol = one.reference()
        # (a rotated query next to a border of two bf16 values may fall on either side: one
        # bf16 step of it, 2^-7, on few elements; its scores move by 2^-7 of a product's share)
        d = (o.to(F64) - ref).abs()
        assert (d <= 2 * tol + 2e-3).all(), float((d - tol).max())


@KV
@pytest.mark.parametrize("more", [0, 190], ids=["few", "many"])
def test_ranges_that_do_not_hold_together_write_nothing(fp8, more):
    from decode_attention_10_b200 import mfa
    b = Batch([2, 3, 4, 2 + more], [50, 60, 0, 200], fp8, 64, seed=10, spare=200)
    rope, pair_axis = make_rope()
    k, v = new_rows(b.rows, 10)
    cache, ws = b.cache(), mfa.Workspace(4)
    n, before = b.rows, snapshot(b)
    for starts in ([0, 2, 5, 9, n + 29], [-3, 2, 5, 9, n], [0, 2, 1, 4, n], [0, 2, 5, n + 900, n],
                   [0, 2, 5, 9, n + 1], [1, 0, 5, 9, n], [0, n, n, n, n - 1]):
        q_start = torch.tensor(starts, dtype=torch.int32, device="cuda")
        q_out = torch.full_like(b.q, 9.0)
        mfa.rope_append(b.q, k, v, cache, q_start, b.seq_lens, rope, q_out=q_out, ws=ws)
        assert mfa.get_error(ws) == 1 and (q_out == 9.0).all(), starts
        mfa.rope_append(None, k, v, cache, q_start, b.seq_lens, ws=ws)
        assert mfa.get_error(ws) == 1, starts
        assert all(torch.equal(x, y) for x, y in zip(snapshot(b), before)), starts
    q_out = mfa.rope_append(b.q, k, v, cache, b.q_start, b.seq_lens, rope, ws=ws)
    assert mfa.get_error(ws) == 0
    verify(b, before, q_out, k, v, rope, pair_axis, None)


def test_a_bad_range_behind_many_sequences_is_seen():
    from decode_attention_10_b200 import mfa
    for more in (0, 300):  # (both kernels; the last range is a later round of a block's threads)
        b = Batch([more] + [0] * 1022 + [3], [0] + [5] * 1023, False, 64, seed=11, spare=8)
        k, v = new_rows(b.rows, 11)
        cache, ws, before = b.cache(), mfa.Workspace(1024), snapshot(b)
        q_start = b.q_start.clone()
        q_start[1024] += 1
        mfa.rope_append(None, k, v, cache, q_start, b.seq_lens, ws=ws)
        assert mfa.get_error(ws) == 1
        assert all(torch.equal(x, y) for x, y in zip(snapshot(b), before))


# Appends of more tokens than SMs run with fewer threads a block, each with more heads: the same
# forms on both sides of that choice.
ROWS = pytest.mark.parametrize("rows", [148, 149, 401])


@KV
@ROWS
@pytest.mark.parametrize("page", [0, 64], ids=["buffers", "p64"])
@pytest.mark.parametrize("rot,axes,interleaved", [(256, 1, False), (256, 3, True), (64, 2, False),
                                                  (208, 4, True), (16, 1, True), (96, 3, False)])
def test_rotated_append_of_few_and_many_tokens(fp8, rows, page, rot, axes, interleaved):
    from decode_attention_10_b200 import mfa
    new = [1, 0, rows - 75, 70, 3, 1]
    b = Batch(new, [64, 9, 100, 0, 31, 255], fp8, page, seed=rot + axes, spare=3)
    rope, pair_axis = make_rope(rot, axes, interleaved)
    k, v = new_rows(rows, rot)
    positions = None
    if axes > 1:
        positions = torch.randint(0, 4096, (axes, rows), dtype=torch.int32, device="cuda",
                                  generator=torch.Generator("cuda").manual_seed(2))
        positions[:, 0], positions[:, rows - 1] = 0, 4095
    before = snapshot(b)
    ws = mfa.Workspace(b.batch)
    q_out = mfa.rope_append(b.q, k, v, b.cache(), b.q_start, b.seq_lens, rope, positions, ws=ws)
    assert mfa.get_error(ws) == 0
    verify(b, before, q_out, k, v, rope, pair_axis, positions)


@KV
@ROWS
@pytest.mark.parametrize("rot", [256, 128])
def test_in_place_and_append_only_of_few_and_many_tokens(fp8, rows, rot):
    from decode_attention_10_b200 import mfa
    b = Batch([rows - 2, 2], [30, 200], fp8, 64, seed=rot)
    rope, _ = make_rope(rot)
    k, v = new_rows(rows, 2)
    want = mfa.rope_append(b.q, k, v, b.cache(), b.q_start, b.seq_lens, rope)
    appended = [b.stored(which, i)[b.cached[i]:].view(torch.uint8).clone()
                for which in "kv" for i in range(2)]
    q = b.q.clone()
    assert mfa.rope_append(q, k, v, b.cache(), b.q_start, b.seq_lens, rope, q_out=q) is q
    assert torch.equal(q, want)
    for buf in (b.k, b.v):
        buf.view(torch.uint8)[:] = 0
    assert mfa.rope_append(None, k, v, b.cache(), b.q_start, b.seq_lens, rope) is None
    again = [b.stored(which, i)[b.cached[i]:].view(torch.uint8) for which in "kv" for i in range(2)]
    assert all(torch.equal(x, y) for x, y in zip(again, appended))


@KV
@ROWS
def test_append_without_rotation_of_few_and_many_tokens(fp8, rows):
    from decode_attention_10_b200 import mfa
    b = Batch([rows - 66, 66], [61, 0], fp8, 64, seed=5)
    k, v = new_rows(rows, 5, ld=520)
    mfa.rope_append(None, k, v, b.cache(), b.q_start, b.seq_lens)
    for i in range(2):
        part = slice(b.starts[i], b.starts[i + 1])
        for which, src, s in (("k", k, b.k_scale), ("v", v, b.v_scale)):
            got = b.stored(which, i)[b.cached[i]:]
            if fp8:
                want = (src[part].float() / s).clamp(-448, 448).to(torch.float8_e4m3fn)
                assert torch.equal(got.view(torch.uint8), want.view(torch.uint8))
            else:
                assert torch.equal(got, src[part])


@KV
@ROWS
def test_rows_of_no_sequence_stay_with_few_and_many_tokens(fp8, rows):
    from decode_attention_10_b200 import mfa
    b = Batch([2, rows - 7], [10, 70], fp8, 64, seed=6, lead=1, behind=4)
    rope, pair_axis = make_rope()
    k, v = new_rows(rows, 6)
    before = snapshot(b)
    q_out = torch.full_like(b.q, 9.0)
    mfa.rope_append(b.q, k, v, b.cache(), b.q_start, b.seq_lens, rope, q_out=q_out)
    verify(b, before, q_out, k, v, rope, pair_axis, None)
    assert (q_out[:1] == 9.0).all() and (q_out[b.starts[-1]:] == 9.0).all()


@KV
@ROWS
def test_bad_tokens_write_nothing_among_few_and_many(fp8, rows):
    from decode_attention_10_b200 import mfa
    b = Batch([2, rows - 2], [62, 60], fp8, 64, seed=7)
    rope, pair_axis = make_rope(rot=128, axes=2, interleaved=True, max_pos=1000)
    k, v = new_rows(rows, 7)
    cache, ws = b.cache(), mfa.Workspace(2)
    good = torch.arange(rows, dtype=torch.int32, device="cuda").repeat(2, 1).contiguous()

    def call(lens=None, positions=good):
        q_out = torch.full_like(b.q, 9.0)
        mfa.rope_append(b.q, k, v, cache, b.q_start, b.seq_lens if lens is None else lens, rope,
                        positions, q_out=q_out, ws=ws)
        return (q_out == 9.0).flatten(1).all(1).nonzero().flatten().tolist(), mfa.get_error(ws)

    assert call() == ([], 0)
    cap = b.per_seq[1] * 64
    # the second sequence ends two past its pages, or begins three before its first row
    assert call(lens=torch.tensor([64, cap + 2], dtype=torch.int32, device="cuda")) == \
        ([rows - 2, rows - 1], 3)
    assert call(lens=torch.tensor([64, rows - 5], dtype=torch.int32, device="cuda")) == ([2, 3, 4], 3)
    for axis, row, p in ((0, 1, -1), (1, rows - 1, 1000), (0, rows - 2, 2 ** 31 - 1), (1, 0, -2 ** 31)):
        pos = good.clone()
        pos[axis, row] = p
        assert call(positions=pos) == ([row], 3)
    before, old = snapshot(b), b.table.clone()
    page = (60 + 40) // 64  # holds positions 64 .. 127 of the second sequence
    for bad in (10 ** 6, -1):
        b.table[1, page] = bad
        lost, err = call()
        assert err == 3 and lost == list(range(2 + 64 - 60, 2 + min(128 - 60, rows - 2)))
        b.table.copy_(old)
        assert all(torch.equal(x, y) for x, y in zip(snapshot(b), before))  # (the others' as before)
