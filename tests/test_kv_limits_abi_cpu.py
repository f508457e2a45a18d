"""Overlapping arguments of the page plan are refused on the host (no GPU)."""
import pytest


@pytest.fixture(scope="module")
def L():
    import block_quantized_decode_quantize_gb300 as m
    from block_quantized_decode_quantize_gb300 import build
    build.build()
    return m.lib()


def test_plan_overlaps(L):
    base, names = 0x7f0000000000, ("ctx", "new", "free", "head", "table", "kv", "cu", "slots", "pos", "out", "st")
    at = {n: base + 4096 * i for i, n in enumerate(names)}       # never dereferenced

    def call(**kw):
        v = dict(at, **kw)
        return L.memra_kv_plan(v["ctx"], v["new"], 3, 16, v["free"], 8, v["head"], v["table"], 2, 6, v["kv"], v["cu"],
                               v["slots"], v["pos"], v["out"], v["st"], None)

    for name, other, words in (("kv", "ctx", 1), ("kv", "ctx", -1), ("kv", "new", 2), ("kv", "free", 0), ("cu", "new", 0),
                               ("cu", "kv", 2), ("slots", "cu", 3), ("pos", "slots", 5), ("pos", "slots", 0), ("out", "ctx", 0),
                               ("out", "table", 5), ("st", "out", 0), ("st", "free", 7), ("table", "free", 7), ("table", "head", -5)):
        assert call(**{name: at[other] + 4 * words}) == 1, (name, other, words)
    assert call(out=at["kv"]) == 1 and call(kv=at["head"]) == 1 and call(out=at["head"], st=at["head"]) == 1


def test_attention_lengths_next_to_2_31(L):
    """A tile of 128 keys beyond the longest sequence must still have 32-bit positions."""
    A = 0x7f0000000000

    def call(max_pages, P):
        return L.memra_kv_attention_q8(A, 0, 2, 4, 256, 64, A, A, A, A, 4, 2, P, 64, 16, A, 2, max_pages, A, A, 1.0, 0, A, A, A,
                                       None, None)

    assert call((2 ** 31 - 1) // 16, 16) == 3 and call((2 ** 31 - 1 - 128) // 16 + 1, 16) == 3
    assert call((2 ** 31 - 1) // 1024 + 1, 1024) == 3
