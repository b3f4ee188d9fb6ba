"""What the paged-cache calls refuse before any launch, and the host plan of the
rotation (no GPU needed)."""
import ctypes

import numpy as np
import pytest

import medusa_head_speculative_heads_gb300 as mg
from medusa_head_speculative_heads_gb300 import paged
from oracle import paged as ref

torch = pytest.importorskip("torch")
# made-up device addresses: only where no GPU could be launched on them
if torch.cuda.is_available():
    pytest.skip("host-validation checks with made-up device pointers run where no GPU is visible", allow_module_level=True)

INVALID, UNSUPPORTED, ALIAS, CUDA, WORKSPACE = 1, 2, 3, 4, 5
F = ctypes.c_float


@pytest.fixture(scope="module", autouse=True)
def built():
    mg.build()


def at(n):
    return (n + 1) << 28  # buffers 256 MiB apart


def plan(r=64, **kw):
    return mg.RopeSpec(r, **kw).ref


@pytest.mark.parametrize("kw", [dict(), dict(scaling="linear", factor=3.0), dict(scaling="bands", base=5e5, factor=8.0, original_len=8192),
                                dict(scaling="ramp", factor=16.0, high=32.0), dict(base=0.5)])
def test_a_plan_holds_the_fractions_of_a_turn(kw):
    st = mg.RopeSpec(96, interleaved=True, magnitude=1.5, **kw).st
    assert (st.rotary_dim, st.interleaved, st.magnitude) == (96, 1, 1.5)
    turns = ref.rope_frequencies(96, **kw) / (2 * np.pi)
    got = np.array([float(t) / 2.0 ** 64 for t in st.turn[:48]])
    # a few roundings of the frequency, and of the fraction itself
    assert np.all(np.abs(got - turns % 1.0) <= 8 * 2.0 ** -53 * np.maximum(turns, 1e-3) + 2.0 ** -60)
    assert not any(st.turn[48:])


@pytest.mark.parametrize("kw", [dict(r=0), dict(r=3), dict(r=258), dict(base=0.0), dict(base=float("inf")), dict(magnitude=float("nan")),
                                dict(scaling="linear", factor=0.0), dict(scaling="bands", low=4.0, high=4.0), dict(scaling="bands", low=0.0),
                                dict(scaling="ramp", base=1.0), dict(scaling="ramp", original_len=0)])
def test_a_plan_refuses(kw):
    kw = dict(kw)
    with pytest.raises(mg.MedusaError):
        mg.RopeSpec(kw.pop("r", 64), **kw)
    with pytest.raises(ValueError):
        mg.RopeSpec(64, scaling="other")


def rope(**o):
    a = dict(q=at(0), ldq=8 * 64, k=at(1), ldk=2 * 64, pos=at(2), plan=plan(), inv=0, nl=2, T=10, hq=8, hkv=2, d=64, dt=1, qo=at(3), ko=at(4))
    a.update(o)
    return mg.lib().medusa_rope(a["q"], a["ldq"], a["k"], a["ldk"], a["pos"], a["plan"], a["inv"], a["nl"], a["T"], a["hq"], a["hkv"], a["d"],
                                a["dt"], a["qo"], a["ko"], None)


@pytest.mark.parametrize("o", [dict(q=None), dict(qo=None), dict(pos=None), dict(plan=None), dict(k=None), dict(ko=None), dict(nl=0), dict(T=0), dict(hq=0),
                               dict(hkv=0), dict(d=62), dict(d=63), dict(d=258), dict(dt=2), dict(ldq=8 * 64 - 1), dict(ldk=127), dict(q=at(0) + 1),
                               dict(pos=at(2) + 2), dict(nl=1 << 16, T=1 << 16)])
def test_rope_refuses(o):
    assert rope(**o) == INVALID


@pytest.mark.parametrize("o", [dict(qo=at(0) + 16), dict(qo=at(0), ldq=1024), dict(ko=at(0) + 64), dict(ko=at(3) + 64), dict(qo=at(2)), dict(ko=at(1) + 2)])
def test_rope_refuses_overlaps(o):
    assert rope(**o) == ALIAS


def append(**o):
    a = dict(q=at(0), ldq=8 * 64, k=at(1), ldk=128, v=at(2), ldv=128, pos=None, plan=plan(), table=at(3), q0=at(4), pl=at(5), nl=2, T=10, B=2, hq=8, hkv=2,
             d=64, np=20, ps=16, mp=8, dt=1, qo=at(6), kp=at(7), vp=at(8))
    a.update(o)
    return mg.lib().medusa_paged_append(a["q"], a["ldq"], a["k"], a["ldk"], a["v"], a["ldv"], a["pos"], a["plan"], a["table"], a["q0"], a["pl"], a["nl"], a["T"],
                                        a["B"], a["hq"], a["hkv"], a["d"], a["np"], a["ps"], a["mp"], a["dt"], a["qo"], a["kp"], a["vp"], None, None)


@pytest.mark.parametrize("o", [dict(k=None), dict(v=None), dict(q=None), dict(qo=None), dict(table=None), dict(q0=None), dict(pl=None), dict(kp=None), dict(B=0),
                               dict(T=0), dict(hkv=0), dict(np=0), dict(ps=0), dict(mp=0), dict(mp=1 << 28), dict(np=1 << 27), dict(ldk=127), dict(ldv=64), dict(dt=5),
                               dict(plan=plan(128)), dict(table=at(3) + 1), dict(d=33)])
def test_append_refuses(o):
    assert append(**o) == INVALID


@pytest.mark.parametrize("o", [dict(vp=at(7) + 1024), dict(k=at(7)), dict(v=at(8) + 64), dict(qo=at(7)), dict(q=at(8)), dict(qo=at(0), ldq=2048), dict(qo=at(1))])
def test_append_refuses_overlaps(o):
    assert append(**o) == ALIAS


def attn(**o):
    a = dict(q=at(0), ldq=8 * 64, kp=at(1), vp=at(2), table=at(3), q0=at(4), pl=at(5), nl=2, T=10, B=2, hq=8, hkv=2, d=64, np=20, ps=16, mp=8, scale=0.1, dt=1,
             out=at(6), lse=at(7), ws=at(8), n=1 << 27)
    a.update(o)
    return mg.lib().medusa_paged_attention(a["q"], a["ldq"], a["kp"], a["vp"], a["table"], a["q0"], a["pl"], a["nl"], a["T"], a["B"], a["hq"], a["hkv"], a["d"], a["np"],
                                           a["ps"], a["mp"], F(a["scale"]), a["dt"], a["out"], a["lse"], a["ws"], a["n"], None, None)


BAD = [dict(q=None), dict(kp=None), dict(vp=None), dict(table=None), dict(pl=None), dict(out=None), dict(B=0), dict(hq=7), dict(hkv=0), dict(d=66), dict(d=0), dict(d=260),
       dict(np=0), dict(ps=0), dict(mp=1 << 29), dict(scale=0.0), dict(scale=float("inf")), dict(scale=float("nan")), dict(dt=3), dict(q=at(0) + 8), dict(out=at(6) + 4),
       dict(kp=at(1) + 2), dict(lse=at(7) + 2), dict(pl=at(5) + 1), dict(nl=0), dict(np=1 << 30)]


@pytest.mark.parametrize("o", BAD + [dict(q0=None), dict(T=0), dict(ldq=511), dict(ldq=518)])
def test_chunk_attention_refuses(o):
    assert attn(**o) == INVALID


@pytest.mark.parametrize("o", [dict(out=at(0)), dict(out=at(1) + 16), dict(lse=at(6) + 8), dict(lse=at(2)), dict(lse=at(0))])
def test_chunk_attention_refuses_overlaps(o):
    assert attn(**o) == ALIAS


def tree(**o):
    a = dict(q=at(0), kp=at(1), vp=at(2), table=at(3), kt=at(4), vt=at(5), mask=at(6), pl=at(7), nl=2, B=2, N=10, hq=8, hkv=2, d=64, np=20, ps=16, mp=8, scale=0.1,
             dt=1, out=at(8), lse=None, ws=at(9), n=1 << 27)
    a.update(o)
    return mg.lib().medusa_paged_tree_attention(a["q"], a["kp"], a["vp"], a["table"], a["kt"], a["vt"], a["mask"], a["pl"], a["nl"], a["B"], a["N"], a["hq"], a["hkv"], a["d"],
                                                a["np"], a["ps"], a["mp"], F(a["scale"]), a["dt"], a["out"], a["lse"], a["ws"], a["n"], None, None)


@pytest.mark.parametrize("o", [x for x in BAD if not set(x) & {"lse", "pl", "out"}] + [dict(out=at(8) + 4), dict(lse=at(10) + 2), dict(pl=None), dict(mask=None),
                               dict(mask=at(6) + 2), dict(kt=None), dict(vt=at(5) + 8), dict(N=0), dict(N=257)])
def test_tree_attention_refuses(o):
    assert tree(**o) == INVALID


def test_tree_attention_refuses_overlaps_and_short_workspaces():
    assert tree(out=at(0)) == ALIAS and tree(out=at(4) + 16) == ALIAS and tree(lse=at(5)) == ALIAS and tree(lse=at(8) + 64) == ALIAS
    need = mg.lib().medusa_paged_attention_workspace_size(2, 20, 2, 8, 2, 64, 16, 1)
    assert need > 0 and need == mg.lib().medusa_paged_attention_workspace_size(7, 20, 2, 8, 2, 64, 16, 1)
    for call in (tree, attn):
        assert call(ws=None) == WORKSPACE and call(n=64) == WORKSPACE and call(ws=at(11) + 8) == WORKSPACE
    assert tree(n=need - 1) == WORKSPACE
    for bad in ((0, 1, 1, 1, 1, 64, 16, 1), (1, 1, 1, 3, 2, 64, 16, 1), (1, 1, 1, 1, 1, 64, 0, 1), (1, 1, 1, 1, 1, 64, 16, 9)):
        assert mg.lib().medusa_paged_attention_workspace_size(*bad) == 0


def compact(**o):
    a = dict(kp=at(0), vp=at(1), table=at(2), kt=at(3), vt=at(4), path=at(5), acc=at(6), pl=at(7), nl_=at(8), nl=2, B=2, N=10, hkv=2, d=64, np=20, ps=16, mp=8, D=4, dt=1)
    a.update(o)
    return mg.lib().medusa_paged_compact(a["kp"], a["vp"], a["table"], a["kt"], a["vt"], a["path"], a["acc"], a["pl"], a["nl_"], a["nl"], a["B"], a["N"], a["hkv"], a["d"],
                                         a["np"], a["ps"], a["mp"], a["D"], a["dt"], None, None)


@pytest.mark.parametrize("o", [dict(kp=None), dict(vt=None), dict(path=None), dict(acc=None), dict(nl_=None), dict(B=0), dict(N=0), dict(N=257), dict(d=0), dict(d=257),
                               dict(D=-1), dict(D=17), dict(np=0), dict(ps=0), dict(mp=0), dict(dt=2), dict(kt=at(3) + 1), dict(path=at(5) + 2), dict(nl=1 << 28)])
def test_compaction_refuses(o):
    assert compact(**o) == INVALID


@pytest.mark.parametrize("o", [dict(vp=at(0)), dict(kt=at(0) + 16), dict(vt=at(1)), dict(nl_=at(7) + 4), dict(nl_=at(6)), dict(nl_=at(5) + 8), dict(nl_=at(2))])
def test_compaction_refuses_overlaps(o):
    assert compact(**o) == ALIAS


@pytest.mark.parametrize("call,o", [
    (append, dict(qo=at(3))), (append, dict(q0=at(7) + 64)), (append, dict(pl=at(8))), (append, dict(pos=at(6) + 4)), (append, dict(table=at(7))),
    (attn, dict(out=at(3))), (attn, dict(lse=at(4))), (attn, dict(out=at(5))), (attn, dict(ws=at(0))), (attn, dict(ws=at(1) + 64)), (attn, dict(ws=at(6))),
    (attn, dict(ws=at(7))), (attn, dict(table=at(8) + 256)), (tree, dict(out=at(6))), (tree, dict(ws=at(5))), (tree, dict(ws=at(7))), (tree, dict(lse=at(9))),
    (compact, dict(nl_=at(0))), (compact, dict(nl_=at(4) + 8)), (compact, dict(path=at(1))), (compact, dict(pl=at(0), nl_=at(0))), (compact, dict(table=at(1) + 16))])
def test_tables_lengths_and_workspaces_may_not_overlap_what_is_written(call, o):
    assert call(**o) == ALIAS


def test_the_binding_refuses_other_shapes_types_and_places():
    i32, bf = torch.int32, torch.bfloat16
    z = lambda *s, dt=bf: torch.zeros(*s, dtype=dt)  # noqa: E731
    spec = mg.RopeSpec(32)
    with pytest.raises(ValueError):  # not on a GPU
        mg.medusa_rope(z(1, 2, 4, 32), z(1, 2, 4, 32), z(2, dt=i32), spec)
    with pytest.raises(ValueError):
        mg.medusa_paged_attention(z(1, 2, 4, 32), z(1, 3, 8, 2, 32), z(1, 3, 8, 2, 32), z(1, 2, dt=i32), z(2, dt=i32), z(1, dt=i32))
    with pytest.raises(TypeError):  # no kernel for fp16
        mg.medusa_rope(z(1, 2, 4, 32, dt=torch.float16), None, z(2, dt=i32), spec)
    stride = paged._token_stride
    assert stride("x", "q", z(2, 5, 6, 32)[:, :, :4], 2, 5, 4, 32) == 192 and stride("x", "q", z(2, 1, 6, 32)[:, :, :4], 2, 1, 4, 32) == 192
    for t, dims in ((z(2, 5, 4, 64)[..., ::2], (2, 5, 4, 32)), (z(2, 4, 5, 32).transpose(1, 2), (2, 5, 4, 32)), (z(2, 6, 4, 32)[:, :5], (2, 5, 4, 32)),
                    (z(2, 5, 4, 32), (2, 5, 4, 64))):
        with pytest.raises(ValueError):
            stride("x", "q", t, *dims)
