"""The build's own care: what a compiler that fails or is killed leaves behind is
never taken for a finished object file."""
import os
import stat

import pytest


def test_partial_objects_are_not_kept(tmp_path, monkeypatch):
    from quantized_attention_08_b200 import build
    broken = tmp_path / "nvcc"
    # writes a part of its output, then dies without a word
    broken.write_text('#!/bin/sh\nwhile [ $# -gt 0 ]; do [ "$1" = -o ] && echo part > "$2"; shift; done\nexit 1\n')
    broken.chmod(broken.stat().st_mode | stat.S_IXUSR)
    monkeypatch.setattr(build, "_nvcc", lambda: str(broken))
    monkeypatch.setattr(build, "OBJ", str(tmp_path / "objects"))
    for _ in range(2):  # the second time nothing may look up to date
        with pytest.raises(RuntimeError, match="building .*cu failed"):
            build._objects(False, False)
        assert os.listdir(tmp_path / "objects") == []
