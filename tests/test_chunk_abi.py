"""The chunk calls without a GPU: arguments that are refused before any device work, table and
workspace sizes, and the plain forms that the GPU tests compare with."""

import ctypes
import math

import pytest
import torch

import chunk_util as cu
from decode_attention_10_b200 import mfa
from oracle import mfa as omfa

P = ctypes.c_void_p
FAKE = P(4096)  # never dereferenced: every call below fails its checks on the host
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    from decode_attention_10_b200 import build
    build.build()
    return mfa.load()


def kv(batch=4, dtype=0, k=1.0, v=1.0, table=4096, page=0):
    return ctypes.byref(mfa.KvCacheDesc(batch, dtype, k, v, table, page))


def test_table_sizes(lib):
    assert lib.mfa_chunk_table_bytes(0) == 0 == lib.mfa_chunk_table_bytes(mfa.MAX_BATCH + 1)
    for b in (1, 16, mfa.MAX_BATCH):
        assert lib.mfa_chunk_table_bytes(b) == lib.mfa_kv_table_bytes(b) + 256 * b
    assert lib.mfa_chunk_workspace_bytes(0) == 0 == lib.mfa_chunk_workspace_bytes(1025)


def test_chunk_attention_refusals(lib):
    def call(q=FAKE, c=None, starts=FAKE, lens=FAKE, n=5, scale=0.0625, out=P(1 << 30), ws=FAKE,
             size=BIG):
        return lib.mfa_chunk_attn(q, c if c is not None else kv(), starts, lens, n, scale, out,
                                  ws, size, None)

    for bad in (dict(q=None), dict(q=P(4104)), dict(out=None), dict(out=P(4100)),
                dict(starts=None), dict(starts=P(4098)), dict(lens=None), dict(lens=P(4097)),
                dict(n=0), dict(n=-1), dict(n=mfa.MAX_ROWS + 1), dict(scale=0.0),
                dict(scale=-1.0), dict(scale=math.nan), dict(scale=math.inf), dict(scale=1e-40),
                dict(out=FAKE),
                dict(out=P(4096 + 5 * 32768 - 16)), dict(q=P((1 << 30) + 16)), dict(ws=None),
                dict(ws=P(4096 + 16)),
                dict(c=kv(batch=0)), dict(c=kv(batch=1025)), dict(c=kv(table=None)),
                dict(c=kv(table=4096 + 64)), dict(c=kv(page=96)), dict(c=kv(page=32)),
                dict(c=kv(dtype=1, k=0.0)), dict(c=kv(dtype=1, v=-1.0))):
        assert call(**bad) == 1, bad
    assert lib.mfa_chunk_attn(FAKE, None, FAKE, FAKE, 5, 0.0625, FAKE, FAKE, BIG, None) == 1
    assert call(c=kv(dtype=2)) == 2


def test_rope_append_refusals(lib):
    def rope(table=4096, max_pos=10, rot=256, inter=0, axes=1, pair=0):
        return mfa.RopeDesc(table, max_pos, rot, inter, axes, (ctypes.c_uint8 * 128)(*[pair] * 128))

    def call(q=FAKE, k=FAKE, k_ld=256, v=FAKE, v_ld=256, r=rope(), pos=None, c=None,
             starts=FAKE, lens=FAKE, n=5, out=FAKE, ws=FAKE):
        return lib.mfa_rope_append(q, k, k_ld, v, v_ld, ctypes.byref(r) if r else None, pos,
                                   c if c is not None else kv(), starts, lens, n, out, ws, BIG,
                                   None)

    for bad in (dict(k=None), dict(k=P(4100)), dict(v=None), dict(v=P(4104)), dict(k_ld=255),
                dict(k_ld=260), dict(v_ld=128), dict(v_ld=257), dict(q=None), dict(out=None),
                dict(q=P(4104)), dict(out=P(4104)), dict(out=P(4112)), dict(q=P(5 * 32768)),
                dict(starts=None), dict(lens=None),
                dict(starts=P(4098)), dict(n=0), dict(n=mfa.MAX_ROWS + 1), dict(r=None),
                dict(r=rope(table=None)), dict(r=rope(table=4100)), dict(r=rope(max_pos=0)),
                dict(r=rope(rot=0)), dict(r=rope(rot=8)), dict(r=rope(rot=24)),
                dict(r=rope(rot=272)), dict(r=rope(axes=0)), dict(r=rope(axes=5), pos=FAKE),
                dict(r=rope(axes=2)),  # several axes need positions
                dict(r=rope(axes=2, pair=2), pos=FAKE), dict(pos=P(4097)), dict(ws=None),
                dict(c=kv(batch=0)), dict(c=kv(dtype=1, k=0.0)),
                dict(q=None, out=None, r=None, pos=FAKE)):
        assert call(**bad) == 1, bad
    assert call(c=kv(dtype=9)) == 2


def far_rope():
    return type("R", (), {"addr": 4096, "n_axes": 1, "device_index": 1})()


def test_binding_refusals(lib):
    # (a workspace and a cache that no call gets as far as using)
    ws = type("W", (), {"addr": 4096, "nbytes": BIG, "device_index": 0})()
    desc = mfa.KvCacheDesc(2, 0, 1.0, 1.0, 4096, 0)
    cache = type("C", (), {"batch": 2, "addr": ctypes.addressof(desc), "device_index": 0})()
    starts, lens = torch.zeros(3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    q = torch.zeros(4, 64, 256, dtype=torch.bfloat16)
    kv = torch.zeros(4, 512, dtype=torch.bfloat16)
    k, v = kv[:, :256], kv[:, 256:]
    with pytest.raises(ValueError, match="q: expected a CUDA tensor"):
        mfa.chunk_attn(q, cache, starts, lens, out=q, ws=ws)
    with pytest.raises(ValueError, match="k: expected a CUDA tensor"):
        mfa.rope_append(q, k, v, cache, starts, lens, ws=ws)
    with pytest.raises(ValueError, match="q_out without q"):
        mfa.rope_append(None, k, v, cache, starts, lens, q_out=q, ws=ws)
    with pytest.raises(TypeError, match="k must be a tensor"):
        mfa.rope_append(None, type("K", (), {"shape": (4,)})(),
                        v, cache, starts, lens, ws=ws)
    for bad in (q.float(), q[:, :32], q.view(4, 256, 64), q[0]):
        with pytest.raises(ValueError, match="q must be"):
            mfa.chunk_attn(bad, cache, starts, lens, out=q, ws=ws)
    for bad in (k.float(), kv[:, :255], kv):
        with pytest.raises(ValueError, match="k must be"):
            mfa.rope_append(None, bad, v, cache, starts, lens, ws=ws)
    # the words for each of the other arguments
    for args, words in ((("v", kv[:, 250:], torch.bfloat16, (4, 256), False), "v must be bfloat16"),
                        (("seq_lens", lens.long(), torch.int32, (2,), True), "seq_lens must be int32"),
                        (("q_start", starts[:2], torch.int32, (3,), True), "q_start must be int32")):
        with pytest.raises(ValueError, match=words):
            mfa._refuse(-1, "", args)
    with pytest.raises(mfa.MfaError, match="MFA_ERR_WORKSPACE"):
        mfa._refuse(4, "x")
    for name, n in (("rope_append", 15), ("chunk_attn", 11), ("bind", 2)):
        with pytest.raises(TypeError):
            getattr(mfa._chunk, name)(*[0] * (n - 1))
    with pytest.raises(ValueError, match="rot_dim"):
        mfa.Rope(torch.zeros(5, 24))
    with pytest.raises(ValueError, match="float32"):
        mfa.Rope(torch.zeros(5, 32, dtype=torch.float64))
    for axes in ([0] * 15, [0] * 15 + [4], [-1] * 16):
        with pytest.raises(ValueError, match="pair_axis"):
            mfa.Rope(torch.zeros(5, 32), axes)
    # memory on several devices
    far = type("W", (), {"addr": 4096, "nbytes": BIG, "device_index": 1})()
    with pytest.raises(ValueError, match="one device"):
        mfa.chunk_attn(q, cache, starts, lens, out=q, ws=far)
    with pytest.raises(ValueError, match="one device"):
        mfa.rope_append(q, k, v, cache, starts, lens, rope=far_rope(), ws=ws)
    # what the binding passes on: a table of the wrong place
    with pytest.raises(ValueError, match="CUDA"):
        mfa.Rope(torch.zeros(5, 32))


def test_rope_table_on_the_cpu():
    t = mfa.rope_table(300, 32, base=500.0, scale=0.5, device="cpu")
    for p in (0, 1, 7, 299):
        for i in range(16):
            ang = 0.5 * p * 500.0 ** (-2 * i / 32)
            assert abs(float(t[p, i]) - math.cos(ang)) <= 2.0 ** -24
            assert abs(float(t[p, 16 + i]) - math.sin(ang)) <= 2.0 ** -24


def test_plain_attention_is_the_oracle_s():
    g = torch.Generator().manual_seed(1)
    q = torch.randn(3, 64, 256, generator=g, dtype=torch.float64)
    k, v = (torch.randn(9, 256, generator=g, dtype=torch.float64) for _ in range(2))
    out, mag, _ = cu.attention(q, k, v, 6, 1 / 16)
    for i in range(3):
        want = omfa.decode_attn_seq(q[i].numpy(), k[:7 + i].numpy(), v[:7 + i].numpy(), 1 / 16)
        assert abs(out[i].numpy() - want).max() < 1e-12
    assert (mag >= out.abs() - 1e-12).all()


@pytest.mark.parametrize("interleaved", [False, True])
def test_plain_rotation_turns_pairs(interleaved):
    # as complex numbers: pair i is multiplied by e^{i angle}; the rest stays
    g = torch.Generator().manual_seed(2)
    x = torch.randn(5, 3, 256, generator=g, dtype=torch.float64)
    ang = torch.randn(5, 24, generator=g, dtype=torch.float64)
    y = cu.rotate(x, ang.cos(), ang.sin(), interleaved)
    for i in range(24):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, 24 + i)
        z = torch.complex(x[..., a], x[..., b]) * torch.polar(torch.ones(5, dtype=torch.float64),
                                                               ang[:, i])[:, None]
        assert (y[..., a] - z.real).abs().max() < 1e-12
        assert (y[..., b] - z.imag).abs().max() < 1e-12
    assert torch.equal(y[..., 48:], x[..., 48:])


def test_rotated_queries_over_the_new_keys_or_values_are_refused(lib):
    rope = mfa.RopeDesc(4096, 10, 256, 0, 1, (ctypes.c_uint8 * 128)())
    q, out, k, v = 1 << 30, 2 << 30, 3 << 30, 4 << 30
    n, ld = 5, 512
    q_bytes, span = n * 64 * 256 * 2, ((n - 1) * ld + 256) * 2

    def call(q=q, out=out, k=k, v=v):
        # (a workspace of no size: a call that passes the checks before it is refused for that,
        # or for the lack of a device)
        return lib.mfa_rope_append(P(q), P(k), ld, P(v), ld, ctypes.byref(rope), None, kv(), FAKE, FAKE,
                                   n, P(out), FAKE, 0, None)

    assert call() in (4, 5) and call(out=q) in (4, 5)
    assert call(k=v - 512) in (4, 5)  # halves of one projection
    for which in ("k", "v"):
        for at in (out, out + 16, out + q_bytes - 16, out - 16, out - span + 16):
            assert call(**{which: at}) == 1, (which, at - out)
        for at in (out + q_bytes, out - span):
            assert call(**{which: at}) in (4, 5)
        assert call(out=q, **{which: q + 32}) == 1  # in place
        assert call(out=out, **{which: q + 32}) in (4, 5)  # (the queries are only read)


def test_decode_calls_need_no_binding(lib, monkeypatch, tmp_path):
    monkeypatch.setattr(mfa, "_lib", None)
    monkeypatch.setattr(mfa, "_chunk", None)
    monkeypatch.setattr(mfa, "BINDING_PATH", str(tmp_path / "mfa_torch.so"))
    assert mfa.load().mfa_version() == lib.mfa_version()
    ws = type("W", (), {"addr": 4096, "nbytes": BIG, "device_index": 0})()
    desc = mfa.KvCacheDesc(2, 0, 1.0, 1.0, 4096, 0)
    cache = type("C", (), {"batch": 2, "addr": ctypes.addressof(desc), "device_index": 0})()
    q = torch.zeros(4, 64, 256, dtype=torch.bfloat16)
    starts, lens = torch.zeros(3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(RuntimeError, match="mfa_torch.so is missing: build it"):
        mfa.chunk_attn(q, cache, starts, lens, out=q, ws=ws)
    (tmp_path / "mfa_torch.so").write_bytes(b"of another torch")
    with pytest.raises(RuntimeError, match="does not fit torch .*build it"):
        mfa.rope_append(None, q, q, cache, starts, lens, ws=ws)


def test_binding_is_built_again_for_another_torch(monkeypatch, tmp_path):
    from decode_attention_10_b200 import build
    monkeypatch.setattr(build, "BINDING", str(tmp_path / "mfa_torch.so"))
    monkeypatch.setattr(build, "BINDING_FOR", str(tmp_path / "built" / "mfa_torch.txt"))
    compiled = []

    def compiler(cmd, check):
        compiled.append(cmd)
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write("binding")

    monkeypatch.setattr(build.subprocess, "run", compiler)
    for version, builds in (("1.0", 1), ("1.0", 1), ("2.0", 2), ("2.0", 2), ("1.0", 3)):
        monkeypatch.setattr(torch, "__version__", version)
        build.build_binding()
        assert len(compiled) == builds, version
    build.os.remove(build.BINDING_FOR)  # (nobody knows what it was built for)
    build.build_binding()
    assert len(compiled) == 4
