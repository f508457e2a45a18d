"""Host-side argument checks of the KV cache, attention and routing entry points (no GPU)."""
import pytest

A = 0x7f0000000000     # never dereferenced: every call below is refused or has no work


@pytest.fixture(scope="module")
def L():
    import block_quantized_decode_quantize_gb300 as m
    from block_quantized_decode_quantize_gb300 import build
    build.build()
    return m.lib()


def test_plan_argument_errors(L):
    def call(ctx=A, new=A, B=2, P=16, free=A, F=4, head=A, table=A, mp=3, T=5, kv=A, cu=A, slots=A,
             pos=A, out=A, st=None):
        return L.memra_kv_plan(ctx, new, B, P, free, F, head, table, mp, T, kv, cu, slots, pos, out, st, None)

    assert call(B=-1) == 1 and call(F=-1) == 1 and call(mp=-1) == 1 and call(T=-1) == 1
    assert call(P=0) == 1 and call(P=24) == 1 and call(P=2048) == 3
    assert call(ctx=None) == 1 and call(table=None) == 1 and call(free=None) == 1
    assert call(slots=None) == 1 and call(cu=None) == 1 and call(out=None) == 1
    for name in ("ctx", "new", "free", "head", "table", "kv", "cu", "slots", "pos", "out", "st"):
        assert call(**{name: A + 2}) == 2, name
    assert call(T=2 ** 31) == 3 and call(B=2 ** 30) == 3


def test_append_and_read_argument_errors(L):
    def call(k=A, v=A, dt=0, T=3, st=128, sh=64, slots=A, kq=A, kd=A, vq=A, vd=A, n=4, H=2, P=16, D=64, S=16,
             status=None):
        return L.memra_kv_append_q8(k, v, dt, T, st, sh, slots, kq, kd, vq, vd, n, H, P, D, S, status, None)

    assert call(T=0) == 0
    assert call(dt=2) == 1 and call(T=-1) == 1 and call(H=0) == 1 and call(n=-1) == 1
    assert call(P=8) == 1 and call(S=0) == 1 and call(S=5) == 1 and call(D=96) == 3 and call(P=1040, S=16) == 3
    assert call(n=2 ** 31) == 3 and call(k=None) == 1 and call(kd=None) == 1 and call(slots=None) == 1
    assert call(k=A + 8) == 2 and call(vq=A + 8) == 2 and call(kd=A + 2) == 2
    assert call(st=132) == 2 and call(sh=4) == 2 and call(dt=1, st=130) == 2

    def read(slots=A, N=3, kq=A, n=4, H=2, P=16, D=64, S=16, dt=0, k=A, v=A):
        return L.memra_kv_read_q8(slots, N, kq, A, A, A, n, H, P, D, S, dt, k, v, None, None)

    assert read(N=0) == 0 and read(N=-1) == 1 and read(dt=7) == 1 and read(k=None) == 1 and read(slots=None) == 1
    assert read(v=A + 4) == 2 and read(D=32) == 3 and read(S=3) == 1


def test_attention_argument_errors(L):
    def call(q=A, dt=0, T=2, Hq=4, st=256, sh=64, kq=A, kd=A, n=4, H=2, P=16, D=64, S=16, table=A, B=2, mp=3,
             lens=A, cu=A, window=0, out=A, lse=A, ws=A):
        return L.memra_kv_attention_q8(q, dt, T, Hq, st, sh, kq, kd, A, A, n, H, P, D, S, table, B, mp, lens, cu, 1.0,
                                       window, out, lse, ws, None, None)

    assert call(T=0) == 0
    assert call(T=-1) == 1 and call(Hq=3) == 1 and call(Hq=0) == 1 and call(H=0) == 1 and call(B=-1) == 1
    assert call(window=-1) == 1 and call(dt=5) == 1 and call(P=20) == 1 and call(S=7) == 1 and call(D=80) == 3
    assert call(q=None) == 1 and call(out=None) == 1 and call(ws=None) == 1 and call(cu=None) == 1
    assert call(lens=None) == 1 and call(table=None) == 1 and call(kd=None) == 1
    assert call(q=A + 8) == 2 and call(ws=A + 8) == 2 and call(st=260) == 2 and call(lse=A + 1) == 2
    assert call(T=2 ** 31) == 3 and call(mp=2 ** 30) == 3


def test_route_argument_errors(L):
    def call(x=A, dt=1, T=2, E=16, st=16, bias=None, score=0, ng=1, tg=1, gt=1, k=4, rn=1, ids=A, w=A):
        return L.memra_moe_route(x, dt, T, E, st, bias, score, ng, tg, gt, k, rn, 1.0, ids, w, None)

    assert call(T=0) == 0
    assert call(T=-1) == 1 and call(E=0) == 1 and call(k=0) == 1 and call(k=17) == 1 and call(dt=2) == 1
    assert call(score=2) == 1 and call(rn=2) == 1 and call(ng=0) == 1 and call(ng=3) == 1 and call(tg=2) == 1
    assert call(ng=16, tg=16, gt=2) == 1 and call(gt=3) == 1 and call(ng=8, tg=1, k=3) == 1
    assert call(E=2048, st=2048) == 3 and call(E=128, k=65) == 3 and call(E=64, ng=64, tg=64) == 3
    assert call(x=None) == 1 and call(ids=None) == 1 and call(x=A + 2) == 2 and call(w=A + 2) == 2
    assert call(bias=A + 1) == 2
