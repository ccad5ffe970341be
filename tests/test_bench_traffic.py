"""The counted HBM bytes that bench.py reports are those of the counter passes
on the sources they are tied to (CPU only): the digest and the numbers stand
beside the counters in profiles/, so that neither changes without the other.
"""
import os
import re
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)
import bench  # noqa: E402


def _profile():
    with open(os.path.join(ROOT, "profiles", "ep_share_32k_hbm_traffic.md")) as f:
        return f.read()


def test_the_digest_is_the_counters_own():
    assert re.findall(r"`sources_sha256` ([0-9a-f]{64})", _profile()) == [bench.TRAFFIC["sources_sha256"]]


def test_the_bytes_are_the_counters_own():
    rows = re.findall(r"^\| `[^`]*` \| (gg_\w+)[^|]* \| (\d+) \| (\d+) \| ([\d.]+) \| ([\d.]+) \|$", _profile(), re.M)
    assert {r[0] for r in rows} == set(bench.TRAFFIC["bytes_per_launch"])
    for name, fetch, write, read_gib, write_gib in rows:
        assert abs(int(fetch) * 2 / 2 ** 20 - float(read_gib)) <= 6e-4
        assert abs(int(write) / 2 ** 20 - float(write_gib)) <= 6e-4
        assert bench.TRAFFIC["bytes_per_launch"][name] == (float(read_gib) + float(write_gib)) * 2 ** 30


def test_other_sources_report_nothing(monkeypatch):
    assert bench.measured_traffic("gg_gateup_fwd", "ep_share_32k") is not None
    monkeypatch.setattr(bench, "TRAFFIC_SOURCES", bench.TRAFFIC_SOURCES[:-1])
    assert bench.measured_traffic("gg_gateup_fwd", "ep_share_32k") is None
