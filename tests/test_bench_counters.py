"""The digest that says whether the stored counter figures belong to the sources here."""
import json
import os
import shutil

import bench

CSRC = os.path.join("stream_residual_mixing_amd", "csrc")


def test_digest_covers_every_source_but_the_uncounted(tmp_path, monkeypatch):
    real = os.path.join(bench.ROOT, CSRC)
    copy = tmp_path / CSRC
    shutil.copytree(real, copy)
    want = bench.source_digest()
    monkeypatch.setattr(bench, "ROOT", str(tmp_path))
    assert bench.source_digest() == want
    for name in sorted(os.listdir(real)):
        text = (copy / name).read_bytes()
        (copy / name).write_bytes(text + b"\n")
        same = bench.source_digest() == want
        assert same == (name in bench.UNCOUNTED_SOURCES), name
        (copy / name).write_bytes(text)
    assert "hc_abi.hip" not in bench.UNCOUNTED_SOURCES  # it chooses the kernels that a call runs
    (copy / "hc_new.hip").write_bytes(b"// a source to come\n")
    assert bench.source_digest() != want


def test_counters_of_other_sources_are_not_reported():
    with open(os.path.join(bench.ROOT, "profiles", "traffic.json")) as f:
        entries = {k: v for k, v in json.load(f).items() if not k.startswith("_")}
    assert entries
    for name, ent in entries.items():
        assert bench.load_counters(name, ent["source_digest"]) == ent
        assert bench.load_counters(name, "another") is None
