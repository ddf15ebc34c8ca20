"""The committed traffic figures say which source they were measured on (CPU only)."""
import hashlib
import json
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "speculative_decoding_verify_sv_gb300", "csrc")


def _entries():
    with open(os.path.join(ROOT, "profiles", "traffic.json")) as f:
        return json.load(f)


@pytest.mark.parametrize("entry", _entries(), ids=lambda e: e["kernel"].split("<")[0] + " " + e["workload"].split(" ")[0])
def test_figures_of_the_current_source_name_its_kernels(entry):
    """A capture prints the kernel with its template arguments: an entry that claims the current source
    has to have as many as the source declares (one carried over from an older source has not)."""
    path = os.path.join(CSRC, entry["source_file"])
    with open(path, "rb") as f:
        data = f.read()
    assert re.fullmatch(r"[0-9a-f]{16}", entry["source_sha"]) and entry["dram_bytes_per_launch"] > 0
    assert os.path.exists(os.path.join(ROOT, entry["summary"]))
    if hashlib.sha256(data).hexdigest()[:16] != entry["source_sha"]:
        return  # an earlier source: the benchmark does not report it
    for name, args in re.findall(r"(\w+)<([^>]*)>", entry["kernel"]):
        declared = re.search(r"template <([^>]*)>\s*__global__[^{;]*?\b%s\s*\(" % name, data.decode())
        assert declared, name
        assert len(args.split(",")) == len(declared.group(1).split(",")), entry["kernel"]
