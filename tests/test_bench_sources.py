"""A capture's figures are used by the bench only while every source that the captured kernel is built from is as it was."""
import os
import re
import shutil

import bench

CSRC = os.path.join(bench.ROOT, "invariant_verify_gb300", "csrc")


def included(name):
    text = open(os.path.join(CSRC, name)).read()
    return {name}.union(*(included(h) for h in re.findall(r'^#include "(\w+\.cuh)"', text, re.M)))


def test_every_header_counts(tmp_path, monkeypatch):
    """A byte more in any of them is another hash; one in a file that the kernel does not include is not."""
    files = included("biv_gemm.cu")
    assert {"biv_common.cuh", "biv_gumbel.cuh", "biv_act.cuh"} < files
    copy = tmp_path / "invariant_verify_gb300" / "csrc"
    shutil.copytree(CSRC, copy, ignore=lambda d, names: [n for n in names if not n.endswith((".cu", ".cuh"))])
    monkeypatch.setattr(bench, "ROOT", str(tmp_path))
    before = bench.kernel_source_sha256()
    for f in sorted(os.listdir(copy)):
        text = (copy / f).read_bytes()
        (copy / f).write_bytes(text + b"\n")
        assert (bench.kernel_source_sha256() != before) == (f in files), f
        (copy / f).write_bytes(text)
    assert bench.kernel_source_sha256() == before
