"""What the 8-bit record operators refuse before a launch, beyond test_cache8_cpu.py."""
import glob
import os
import subprocess

import pytest
import torch

from host_offload_serving_gb300 import _build, cache8, pages
from host_offload_serving_gb300 import hisparse as H

REC = cache8.Records(2, 64, 64, 16)
TURNS = cache8.rotary_turns(32)[0]


def _zeros(*shape, dtype=torch.int32):
    return torch.zeros(*shape, dtype=dtype)


def _pack(**kw):
    k = _zeros(3, 2, 64, dtype=torch.bfloat16)
    a = dict(k=k, v=k, dst=_zeros(3, 256, dtype=torch.uint8), scales=torch.zeros(1, 4, 4), start=_zeros(1),
             max_len=3, stream=0)
    a.update(kw)
    return cache8.pack(REC, a.pop("k"), a.pop("v"), a.pop("dst"), a.pop("scales"), a.pop("start"), **a)


def test_tensors_that_the_gpu_does_not_reach_are_refused():
    """Pageable host tensors, the frequency table as rotary_turns returns it among them."""
    x = _zeros(3, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="is on cpu"):
        cache8.rotate(x, _zeros(3), TURNS, stream=0)
    with pytest.raises(ValueError, match="is on cpu"):
        _pack()
    q = _zeros(2, 1, 4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="is on cpu"):
        cache8.attend(REC, q, _zeros(2, 8), _zeros(2, 8), _zeros(2, 17, 256, dtype=torch.uint8),
                      torch.zeros(2, 4, 4), torch.zeros_like(q), stream=0)
    with pytest.raises(ValueError, match="CUDA device"):
        pages.PagePool(_zeros(1, 4, 64, dtype=torch.uint8), requests=2, max_blocks=2, block_tokens=4)


def test_pack_checks_its_frequency_table():
    for turns in (TURNS.int(), TURNS.float(), torch.cat([TURNS, TURNS])[::2]):
        with pytest.raises(ValueError, match="turns"):
            _pack(turns=turns)


def test_pages_bound_on_blocks():
    """Table rows so long that 32-bit loops over them would wrap."""
    p = H.PagePool(8, 2, 2 ** 30 + 1, 16, 1, 64, 0x1000, 8 * 1024, 1024, 0x1000, 0x1000, 0x1000, None)
    assert H.hisparse_pages_grow(p, 0x1000, 0x1000, 1, None) == H.EBOUND
    assert H.hisparse_pages_fork(p, 0x1000, 0x1000, 0x1000, 1, None) == H.EBOUND
    assert H.hisparse_pages_free(p, 0x1000, 1, None) == H.EBOUND
    assert H.hisparse_pages_compact(p, None) == H.EBOUND


@pytest.mark.parametrize("fails", ["*pages.cu*", "*-shared*"])
def test_a_build_that_fails_leaves_nothing_behind(tmp_path, monkeypatch, fails):
    """One unit does not compile, or the link fails: the objects go, and so does a half-made library."""
    exe = tmp_path / "nvcc"
    exe.write_text('#!/bin/sh\nprev=\nfor a in "$@"; do [ "$prev" = -o ] && : > "$a"; prev=$a; done\n'
                   f'case "$*" in {fails}) exit 1;; esac\n')
    exe.chmod(0o755)
    out = tmp_path / "out" / "lib.so"
    monkeypatch.setattr(_build, "nvcc", lambda: str(exe))
    monkeypatch.setattr(_build, "OUT", str(out))
    with pytest.raises(subprocess.CalledProcessError):
        _build.build(force=True)
    assert os.listdir(out.parent) == []
    assert not glob.glob(os.path.join(_build.PKG, "_build", f"*.{os.getpid()}.*"))
    exe.write_text(exe.read_text().replace("exit 1", "exit 0"))
    _build.build(force=True)
    assert os.listdir(out.parent) == ["lib.so"]


@pytest.mark.parametrize("dst", [
    _zeros(1, 1, 3, 256, dtype=torch.uint8), _zeros(256, dtype=torch.uint8),
    _zeros(1, 3, 256, dtype=torch.uint8).expand(2, 3, 256),
], ids=["four dimensions", "one", "one request's rows for all"])
def test_pack_refuses_rows_that_are_neither_by_token_nor_by_position(dst):
    with pytest.raises(ValueError, match="dst"):
        _pack(dst=dst, scales=torch.zeros(2, 4, 4))
