"""The smoke run covers every operator of the library."""
import pytest

import sgemm_row_major_gb300 as sg


@pytest.mark.gpu
def test_smoke_runs_every_operator(monkeypatch, capsys):
    import __graft_entry__ as entry
    called = set()

    def counted(name):
        f = getattr(sg, name)

        def run(*a, **k):
            called.add(name)
            return f(*a, **k)
        return run
    names = ["sgemm", "matmul_fp8", "quantize_fp8", "rmsnorm_fp8", "rmsnorm_fp8_backward", "moe_fp8"]
    for name in names:
        monkeypatch.setattr(sg, name, counted(name))
    entry.smoke()
    assert called == set(names) and "smoke ok" in capsys.readouterr().out
