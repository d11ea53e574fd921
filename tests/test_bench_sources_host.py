"""The DRAM record of the decode step is void when its kernel changes: every
source file of the library that the kernel's file includes is one of the
hashed ones (include/pa.h, the public declarations, apart)."""
import hashlib
import json
import os
import re

import bench

CSRC = os.path.join(bench.ROOT, "paged_kv_cache_309_gb300", "csrc")


def _closure(name, seen):
    path = os.path.join(CSRC, name)
    if name in seen or not os.path.exists(path):
        return seen
    seen.add(name)
    with open(path) as f:
        for inc in re.findall(r'^\s*#\s*include\s+"([^"]+)"', f.read(), re.M):
            _closure(inc, seen)
    return seen


def test_the_hash_covers_what_the_kernel_is_made_of():
    with open(os.path.join(bench.ROOT, "profiles", "decode_traffic.json")) as f:
        hashed = {os.path.basename(p) for p in json.load(f)["hashed_sources"]}
    assert _closure("decode.cu", set()) == hashed


def test_an_edit_of_any_of_them_voids_the_record(tmp_path, monkeypatch):
    names = sorted(_closure("decode.cu", set()))
    key = ("w", "fused", "bf16")
    for name in (None, *names):
        src = tmp_path / str(name)
        src.mkdir()
        for n in names:
            with open(os.path.join(CSRC, n)) as f:
                (src / n).write_text(f.read())
        (tmp_path / "profiles").mkdir(exist_ok=True)
        monkeypatch.setattr(bench, "ROOT", str(tmp_path))
        kernel = str(src / "decode.cu")
        h = hashlib.sha256()
        for n in ("decode.cu", "pa_internal.cuh"):
            h.update((src / n).read_bytes())
        (tmp_path / "profiles" / "decode_traffic.json").write_text(json.dumps({"records": [dict(
            workload=key[0], step=key[1], kv_dtype=key[2], source_sha256_16=h.hexdigest()[:16],
            dram_bytes_per_decode_call=7)]}))
        assert bench.traffic_record(kernel, *key) == 7
        if name is not None:
            with open(src / name, "a") as f:
                f.write("\n// edited\n")
            assert bench.traffic_record(kernel, *key) is None, name
