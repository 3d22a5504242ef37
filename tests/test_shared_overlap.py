"""moe_shared_ffn refuses an out or workspace that lies in what the call reads (host only)."""
import pytest

from test_shared_ffn import P, call, needs_lib

SIZES = {"gate_a": 2 * 2 * 8 * 64, "gate_b": 2 * 2 * 8 * 32, "up_a": 2 * 2 * 8 * 64, "up_b": 2 * 2 * 8 * 32,
         "down_a": 2 * 2 * 8 * 32, "down_b": 2 * 2 * 8 * 64}    # bytes: two adapters of rank 8, hidden 64, inter 32
OUT = 3 * 64 * 4


@needs_lib
@pytest.mark.parametrize("where", [0x10000, 0x20000, 0x30000])
def test_weights(where):
    """At the start and the end of each matrix (4096 bytes), and reaching into it from before."""
    for bad in (dict(out=where), dict(out=where + 4096 - 16), dict(out=where - OUT + 16), dict(ws=where), dict(ws=where + 4096 - 256)):
        st, msg, _ = call(**bad)
        assert st == 1 and "overlaps the layer" in msg, (bad, st, msg)


@needs_lib
@pytest.mark.parametrize("name", list(P))
def test_adapters(name):
    for bad in (dict(out=P[name]), dict(out=P[name] + SIZES[name] - 16), dict(ws=P[name]), dict(ws=P[name] + SIZES[name] - 256)):
        st, msg, _ = call(pool={}, **bad)
        assert st == 1 and "adapters' weights" in msg, (bad, st, msg)


@needs_lib
@pytest.mark.parametrize("name", ["rank", "scale"])
def test_ranks_and_scales(name):
    for bad in (dict(out=0x500000), dict(out=0x500000 - OUT + 16), dict(ws=0x500000)):
        st, msg, _ = call(pool={name: 0x500000 + (4 if "out" in bad else 0)}, **bad)
        assert st == 1 and "adapters' weights" in msg, (bad, st, msg)
