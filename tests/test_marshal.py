"""The marshalling module is found by what it was compiled against, and calls without it take the ctypes route."""
import os
import sysconfig

import pytest
import torch

import dsa_lightning_indexer_02_b200 as dsa
from dsa_lightning_indexer_02_b200 import build


@pytest.fixture
def unloaded(monkeypatch):
    monkeypatch.setattr(dsa, "_fast", None)
    return monkeypatch


def test_its_name_tells_what_it_was_built_for(unloaded):
    path = build.marshal_path()
    assert sysconfig.get_config_var("SOABI") in path and torch.__version__ in path
    assert dsa._native().__file__ == path and os.path.dirname(path) == os.path.dirname(dsa.__file__)
    unloaded.setattr(torch, "__version__", "0.0.0")
    assert build.marshal_path() != path


def test_a_module_of_another_torch_is_not_loaded(unloaded):
    unloaded.setattr(torch, "__version__", "0.0.0")
    with pytest.warns(RuntimeWarning, match="ctypes"):
        assert dsa._native() is dsa._Ctypes
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="must be a CUDA tensor"):          # the checks and the call as ever, no second warning
        dsa.dsa_rope(x, x.clone(), torch.zeros(16, dtype=torch.float64))


def test_build_marshal_without_a_compiler(unloaded, capsys):
    unloaded.setattr(build.subprocess, "run", lambda *a, **k: (_ for _ in ()).throw(FileNotFoundError("g++")))
    assert build.build_marshal(force=True) is None and "not built" in capsys.readouterr().err


@pytest.mark.gpu
def test_both_routes_give_the_same(cuda_ok, unloaded):
    g = torch.Generator().manual_seed(0)
    bf = lambda *s: torch.randn(s, generator=g).to(torch.bfloat16).cuda()  # noqa: E731
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    q, k, v = bf(2, 8, 128), bf(2, 2, 128), bf(2, 2, 128)
    f = dsa.rope_freqs(128)[0].cuda()

    def run():
        pages = [torch.zeros((4, 16, 2, 128), dtype=torch.float8_e4m3fn, device="cuda") for _ in range(2)]
        scales = [torch.zeros((4, 2), device="cuda") for _ in range(2)]
        table = i32([0, 1], [2, 3])
        r, out = torch.empty_like(q), torch.empty_like(q)
        dsa.dsa_rope(q, r, f, pos=i32(5, 17))
        dsa.dsa_kv_append(k, v, *pages, *scales, table, i32(0, 0), inv_freq=f)
        dsa.dsa_paged_attn(r, *pages, *scales, table, i32(1, 1), 0.1, out)
        assert dsa.sync_status() == dsa.DSA_OK
        return [r, out, *scales] + [p.view(torch.uint8) for p in pages]

    fast = run()
    assert dsa._fast is not dsa._Ctypes
    unloaded.setattr(dsa, "_fast", dsa._Ctypes)
    assert all(torch.equal(a, b) for a, b in zip(fast, run()))
