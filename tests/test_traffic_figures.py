"""bench.py reports a kernel's HBM traffic from profiles/ only while the file was
taken on the present sources of the kernels it times (no GPU)."""
import os
import shutil

import pytest

from combine_moe_route_histogram_amd import profsum as P


@pytest.mark.parametrize("workload", ["longseq", "mixtral"])
@pytest.mark.parametrize("call", ["dispatch_ffn", "ffn_combine", "ffn_bwd", "combine_bwd", "dispatch_bwd"])
def test_traffic_of_the_timed_kernels_is_reported(call, workload):
    got = P.traffic_bytes(call, workload)
    assert got is not None and got > 0


def test_fingerprint_is_of_the_timed_kernels(tmp_path, monkeypatch):
    """Sources of other calls' kernels may change, those of bench.py's may not."""
    pkg = tmp_path / "pkg"
    shutil.copytree(os.path.join(P.PKG, "csrc"), pkg / "csrc")
    shutil.copytree(os.path.join(P.ROOT, "include"), tmp_path / "include")
    monkeypatch.setattr(P, "PKG", str(pkg))
    monkeypatch.setattr(P, "ROOT", str(tmp_path))
    before = P.source_fingerprint()

    def changed(name):
        path = pkg / "csrc" / name
        text = path.read_text()
        path.write_text(text + "\nint added_for_the_test;\n")
        now = P.source_fingerprint()
        path.write_text(text)
        return now != before
    assert not any(changed(n) for n in ("decode.hip", "decode.hpp", "mx.hip"))
    assert all(changed(n) for n in ("gemm.hip", "gemm_tile.hpp", "fused.hip", "bwd.hip", "rows.hip", "route.hip",
                                    "kernels.hpp", "tuning.hip", "moe_api.hip"))
