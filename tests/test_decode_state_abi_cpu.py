"""Host-side argument checks of the norm and rotation, page and log-probability entry points (no GPU)."""
import ctypes

import pytest

A = 0x7f0000000000     # never dereferenced: every call below is refused or has no work
M = 1 << 28            # between arrays, farther than any of them is long


@pytest.fixture(scope="module")
def L():
    import block_quantized_decode_quantize_gb300 as m
    from block_quantized_decode_quantize_gb300 import build
    build.build()
    return m.lib()


def test_rope_argument_errors(L):
    def call(q=A, k=A + M, dt=0, T=3, Hq=4, Hkv=2, D=64, qt=512, qh=64, kt=512, kh=64, qw=None, kw=None, eps=-1.0,
             pos=A + 2 * M, f=A + 3 * M, R=64, lay=0, qo=A + 4 * M, qod=0, qot=256, qoh=64, ko=A + 5 * M, kod=0, kot=128,
             koh=64):
        return L.memra_qk_norm_rope(q, k, dt, T, Hq, Hkv, D, qt, qh, kt, kh, qw, kw, eps, pos, f, R, lay, qo, qod, qot, qoh,
                                    ko, kod, kot, koh, None)

    assert call(T=0) == 0 and call(Hq=0, Hkv=0) == 0
    assert call(T=-1) == 1 and call(Hq=-1) == 1 and call(Hkv=-1) == 1 and call(R=-8) == 1 and call(R=12) == 1 and call(R=72) == 1
    assert call(D=96) == 3 and call(D=32, R=0) == 3 and call(Hq=65536) == 3 and call(T=2 ** 31) == 3
    assert call(dt=2) == 1 and call(qod=-1) == 1 and call(kod=5) == 1 and call(lay=2) == 1 and call(lay=-1) == 1
    assert call(eps=float("nan")) == 1 and call(eps=float("inf")) == 1 and call(qw=A + 6 * M) == 1
    assert call(q=None) == 1 and call(k=None) == 1 and call(qo=None) == 1 and call(ko=None) == 1
    assert call(pos=None) == 1 and call(f=None) == 1
    assert call(q=A + 8) == 2 and call(ko=A + 5 * M + 8) == 2 and call(qt=516) == 2 and call(koh=68, kot=144) == 2
    assert call(pos=A + 2 * M + 2) == 2 and call(f=A + 3 * M + 4) == 2 and call(eps=1e-6, qw=A + 6 * M + 2) == 2
    assert call(qt=-8) == 1 and call(qt=2 ** 62) == 3 and call(kh=2 ** 60) == 3
    # outputs that meet something: their own rows, inputs, each other
    assert call(qoh=32) == 1 and call(qot=192) == 1 and call(kot=0) == 1
    assert call(qo=A) == 1 and call(ko=A) == 1 and call(qo=A + 16, qot=512) == 1 and call(qo=A + 2 * M) == 1
    assert call(ko=A + 4 * M) == 1 and call(qo=A + 3 * M) == 1
    assert call(k=A + 512, ko=A + 512 + 64, kot=512) == 1 and call(k=A + 512, qo=A + 448, qot=512) == 1


def test_rope_in_place_and_side_by_side_pass_the_checks(L):
    """T = 0 is answered before the checks, so a refusal behind them tells that these were passed: a bad alignment is
    found before overlaps, overlaps before the launch, which has no device here (4) or one that would not start."""
    import torch
    if torch.cuda.is_available():
        pytest.skip("would launch")

    def call(**kw):
        a = dict(q=A, k=A + 512, dt=0, T=3, Hq=4, Hkv=2, qt=1024, kt=1024, qo=A + 4 * M, qot=256, ko=A + 512, kot=1024)
        a.update(kw)
        return L.memra_qk_norm_rope(a["q"], a["k"], a["dt"], a["T"], a["Hq"], a["Hkv"], 64, a["qt"], 64, a["kt"], 64, None, None,
                                    -1.0, A + 2 * M, A + 3 * M, 64, 0, a["qo"], a["dt"], a["qot"], 64, a["ko"], a["dt"], a["kot"],
                                    64, None)

    assert call() == 4                                   # K in place within the projection's rows
    assert call(qo=A, qot=1024) == 4                     # Q too
    assert call(qo=A + 1024, qot=1024) == 4              # Q into columns behind K
    assert call(qo=A + 512 + 128, qot=1024) == 1         # and into K's second head


def test_fork_argument_errors(L):
    def call(par=A, pre=None, C=3, lens=A + M, table=A + 2 * M, B=2, mp=4, P=16, refs=A + 3 * M, n=9, lo=A + 4 * M, to=A + 5 * M,
             st=None):
        return L.memra_kv_fork(par, pre, C, lens, table, B, mp, P, refs, n, lo, to, st, None)

    assert call(C=0) == 0
    assert call(C=-1) == 1 and call(B=-1) == 1 and call(mp=-1) == 1 and call(n=-1) == 1 and call(P=0) == 1 and call(P=24) == 1
    assert call(P=2048) == 3 and call(n=2 ** 30) == 3 and call(mp=2 ** 31) == 3 and call(C=2 ** 25) == 3 and call(B=2 ** 20, mp=2 ** 20) == 3
    for name in ("par", "lens", "table", "refs", "lo", "to"):
        assert call(**{name: None}) == 1, name
    for name in ("par", "pre", "lens", "table", "refs", "lo", "to", "st"):
        assert call(**{name: A + 6 * M + 2}) == 2, name
    assert call(lo=A + M) == 1 and call(to=A + 2 * M) == 1 and call(refs=A) == 1 and call(st=A + 5 * M + 8) == 1 and call(pre=A + 4 * M) == 1


def test_unshare_argument_errors(L):
    def call(lens=A, new=A + M, B=2, P=16, refs=A + 2 * M, n=9, free=A + 3 * M, F=9, head=A + 4 * M, table=A + 5 * M, mp=4, no=A + 6 * M,
             src=A + 7 * M, dst=A + 8 * M, tok=A + 9 * M, out=A + 10 * M, st=None):
        return L.memra_kv_unshare(lens, new, B, P, refs, n, free, F, head, table, mp, no, src, dst, tok, out, st, None)

    assert call(B=-1) == 1 and call(F=-1) == 1 and call(P=8) == 1 and call(P=1040) == 3 and call(F=2 ** 31) == 3
    for name in ("lens", "new", "refs", "free", "table", "no", "src", "dst", "tok", "out"):
        assert call(**{name: None}) == 1, name
    for name in ("lens", "new", "refs", "free", "head", "table", "no", "src", "dst", "tok", "out", "st"):
        assert call(**{name: A + 11 * M + 1}) == 2, name
    assert call(no=A) == 1 and call(out=A + 3 * M) == 1 and call(src=A + 8 * M + 4) == 1 and call(table=A + 2 * M) == 1


def test_copy_pages_argument_errors(L):
    def layer(kq=A, kd=A + M, vq=A + 2 * M, vd=A + 3 * M):
        return [kq, kd, vq, vd]

    def call(layers=None, src=A + 4 * M, dst=A + 5 * M, tok=None, N=3, n=9, H=2, P=16, D=64, S=16, st=None, count=None):
        layers = [layer()] if layers is None else layers
        flat = [x for one in layers for x in one]
        array = (ctypes.c_void_p * max(1, len(flat)))(*flat)
        return L.memra_kv_copy_pages(src, dst, tok, N, ctypes.cast(array, ctypes.c_void_p), len(layers) if count is None else count,
                                     n, H, P, D, S, st, None)

    assert call(N=0) == 0 and call(layers=[]) == 0
    assert call(N=-1) == 1 and call(count=-1) == 1 and call(n=-1) == 1 and call(H=0) == 1 and call(P=17) == 1 and call(S=5) == 1
    assert call(D=96) == 3 and call(P=1040, S=16) == 3 and call(H=40000) == 3 and call(n=2 ** 31) == 3 and call(N=2 ** 33) == 3
    assert call(src=None) == 1 and call(dst=None) == 1 and call(layers=[layer(), layer(vd=None)]) == 1
    assert call(src=A + 2) == 2 and call(tok=A + 1) == 2 and call(st=A + 3) == 2
    assert call(layers=[layer(), layer(kq=A + 8)]) == 2 and call(layers=[layer(kd=A + 2)]) == 2
    assert call(src=A + 64) == 1 and call(tok=A + 3 * M) == 1 and call(st=A + M) == 1


def test_release_argument_errors(L):
    def call(lens=A, keep=None, B=2, P=16, table=A + M, mp=4, refs=A + 2 * M, n=9, free=A + 3 * M, F=9, head=A + 4 * M, lo=A + 5 * M,
             out=A + 6 * M, st=None):
        return L.memra_kv_release(lens, keep, B, P, table, mp, refs, n, free, F, head, lo, out, st, None)

    assert call(B=-1) == 1 and call(F=-1) == 1 and call(P=20) == 1 and call(B=2 ** 24, mp=2 ** 10) == 3
    for name in ("lens", "table", "refs", "free", "head", "lo", "out"):
        assert call(**{name: None}) == 1, name
    for name in ("lens", "keep", "table", "refs", "free", "head", "lo", "out", "st"):
        assert call(**{name: A + 7 * M + 2}) == 2, name
    assert call(lo=A + M) == 1 and call(out=A + 3 * M + 4) == 1 and call(free=A + 2 * M) == 1 and call(keep=A + 5 * M) == 1


def test_compact_argument_errors(L):
    def call(lens=A, table=A + M, B=2, mp=4, P=16, n=9, to=A + 2 * M, refs=A + 3 * M, free=A + 4 * M, src=A + 5 * M, dst=A + 6 * M,
             out=A + 7 * M, st=None):
        return L.memra_kv_compact(lens, table, B, mp, P, n, to, refs, free, src, dst, out, st, None)

    assert call(B=-1) == 1 and call(n=-1) == 1 and call(P=1) == 1 and call(n=2 ** 31) == 3
    for name in ("lens", "table", "to", "refs", "free", "src", "dst", "out"):
        assert call(**{name: None}) == 1, name
    for name in ("lens", "table", "to", "refs", "free", "src", "dst", "out", "st"):
        assert call(**{name: A + 8 * M + 2}) == 2, name
    assert call(to=A) == 1 and call(src=A + 6 * M) == 1 and call(refs=A + M) == 1 and call(to=A + M + 4) == 1


def test_logprobs_argument_errors(L):
    def call(x=A, dt=1, T=2, V=100, st=100, tok=A, n=3, lp=A, h=A, ids=A, top=A, status=None):
        return L.memra_token_logprobs(x, dt, T, V, st, tok, n, lp, h, ids, top, status, None)

    assert call(T=0) == 0
    assert call(T=-1) == 1 and call(V=0) == 1 and call(st=-1) == 1 and call(n=-1) == 1 and call(V=2, n=3) == 1 and call(dt=2) == 1
    assert call(V=2 ** 20 + 1) == 3 and call(n=33) == 3 and call(T=2 ** 31) == 3 and call(st=2 ** 58) == 3
    assert call(x=None) == 1 and call(tok=None) == 1 and call(lp=None) == 1 and call(ids=None) == 1 and call(top=None) == 1
    assert call(x=A + 2) == 2 and call(x=A + 1, dt=0) == 2
    for name in ("tok", "lp", "h", "ids", "top", "status"):
        assert call(**{name: A + 2}) == 2, name


def test_binding_refuses_what_is_not_a_tensor_of_the_right_kind():
    """On CPU tensors the long way names the argument."""
    import torch
    import block_quantized_decode_quantize_gb300 as m
    x = torch.zeros(2, 4, 64)
    i = torch.zeros(2, dtype=torch.int32)
    table = torch.zeros(2, 3, dtype=torch.int32)
    with pytest.raises(ValueError, match="q must be"):
        m.memra_qk_norm_rope(x, x)
    with pytest.raises(ValueError, match="lens"):
        m.memra_kv_fork(i, i, table, 16, i)
    with pytest.raises(ValueError, match="lens"):
        m.memra_kv_unshare(i, i, 16, i, i, table)
    with pytest.raises(ValueError, match="lens"):
        m.memra_kv_release(i, 16, table, i, i, i)
    with pytest.raises(ValueError, match="lens"):
        m.memra_kv_compact(i, table, 16, 9)
    with pytest.raises(ValueError, match="caches|kq"):
        m.memra_kv_copy_pages(i, i, [(x, x, x, x)])
    with pytest.raises(ValueError, match="caches"):
        m.memra_kv_copy_pages(i, i, (x, x, x, x))
    with pytest.raises(ValueError, match="logits"):
        m.memra_token_logprobs(torch.zeros(2, 10))
