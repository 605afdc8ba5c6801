"""How the library is compiled."""
import subprocess

import sliding_window_gqa_prefill_b200 as swa


def test_device_code_is_for_sm_100a_and_not_compressed(monkeypatch, tmp_path):
    """Compressed device code is unpacked in the first call of every process."""
    seen = []
    monkeypatch.setattr(subprocess, "run", lambda cmd, **kw: seen.append(cmd))
    monkeypatch.setattr(swa.os, "replace", lambda a, b: None)
    swa.build(force=True)
    swa.build(force=True, debug=True)
    assert len(seen) == 2
    for cmd in seen:
        assert "--no-compress" in cmd and "arch=compute_100a,code=sm_100a" in cmd
    assert "-DSWA_BOUNDS_CHECK" in seen[1]
