"""What the compiled binding of the paged calls does before it looks for a GPU."""
import pytest

import medusa_head_speculative_heads_gb300 as mg

torch = pytest.importorskip("torch")


class Neither:
    def __bool__(self):
        raise RuntimeError("neither true nor false")


@pytest.fixture(scope="module", autouse=True)
def built():
    mg.build()


def test_a_flag_that_is_neither_true_nor_false_is_its_own_error():
    z = lambda *s, dt=torch.bfloat16: torch.zeros(*s, dtype=dt)  # noqa: E731
    i32 = torch.int32
    pools = (z(1, 3, 8, 2, 32), z(1, 3, 8, 2, 32), z(1, 2, dt=i32))
    for flag in (Neither(), torch.zeros(2)):
        with pytest.raises(RuntimeError, match="neither|ambiguous"):
            mg.medusa_rope(z(1, 2, 4, 32), None, z(2, dt=i32), mg.RopeSpec(32), inverse=flag)
        with pytest.raises(RuntimeError, match="neither|ambiguous"):
            mg.medusa_paged_attention(z(1, 2, 4, 32), *pools, z(2, dt=i32), z(1, dt=i32), want_lse=flag)
        with pytest.raises(RuntimeError, match="neither|ambiguous"):
            mg.medusa_paged_tree_attention(z(1, 1, 2, 4, 32), *pools, z(1, 1, 2, 2, 32), z(1, 1, 2, 2, 32), z(2, 1, dt=i32), z(1, dt=i32), want_lse=flag)


def test_a_rotation_that_would_record_a_gradient_refuses_alike():
    z = torch.zeros(1, 2, 4, 32, requires_grad=True)
    for q, k in ((z, None), (z, z), (z.detach(), z)):
        with pytest.raises(ValueError, match="on a GPU"):
            mg.medusa_rope(q, k, torch.zeros(2, dtype=torch.int32), mg.RopeSpec(32))
    with pytest.raises(TypeError, match="must be a tensor"):
        mg.medusa_rope(3, None, torch.zeros(2, dtype=torch.int32), mg.RopeSpec(32))


def test_the_compiled_file_is_of_one_python_torch_and_abi(monkeypatch):
    """Another Python, torch or C++ ABI never takes this one's binding for its own."""
    import sysconfig

    from medusa_head_speculative_heads_gb300.build import binding_path
    here = binding_path()
    suffix = sysconfig.get_config_var("EXT_SUFFIX")
    assert here.endswith(suffix) and torch.__version__ in here
    others = {here}
    with monkeypatch.context() as m:
        m.setattr(sysconfig, "get_config_var", lambda name: suffix.replace("cpython-3", "cpython-9") if name == "EXT_SUFFIX" else None)
        others.add(binding_path())
    with monkeypatch.context() as m:
        m.setattr(torch, "__version__", "0.0.0")
        others.add(binding_path())
    with monkeypatch.context() as m:
        m.setattr(torch._C, "_GLIBCXX_USE_CXX11_ABI", not torch._C._GLIBCXX_USE_CXX11_ABI)
        others.add(binding_path())
    assert len(others) == 4
