"""The counter summaries under profiles/ carry a hash of the sources they were taken
on: it has to change with every file that the timed kernels are compiled and
dispatched from."""
import json
import os

import pytest

import bench


def test_covers_the_timed_kernels_and_their_dispatch():
    files = bench.timed_sources()
    assert {'api.hip', 'api_common.hpp', 'gdn2_launch.hpp', 'gdn2_device.hpp', 'decode.hip', 'chunk.hip',
            'chunk_impl.hpp', 'chunk_bwd_impl.hpp', 'chunk_cs_impl.hpp', 'chunk_bf16_d128.hip'} <= set(files)
    assert not [f for f in files if f.startswith(('recurrent', 'prologue', 'layer_norm', 'operators', 'column_sums'))]


@pytest.mark.parametrize('name', ['gdn2_launch.hpp', 'api.hip', 'decode.hip', 'chunk_bwd_impl.hpp'])
def test_changes_with_each_of_them(name, tmp_path, monkeypatch):
    for f in os.listdir(bench.CSRC):
        with open(os.path.join(bench.CSRC, f), 'rb') as fh:
            (tmp_path / f).write_bytes(fh.read())
    before = bench.src_hash()
    monkeypatch.setattr(bench, 'CSRC', str(tmp_path))
    assert bench.src_hash() == before
    with open(tmp_path / name, 'a') as fh:
        fh.write('\n')
    assert bench.src_hash() != before


@pytest.mark.parametrize('name', ['traffic.json', 'mfma.json'])
def test_summaries_name_their_commit(name):
    """Each summary says which hash and which commit it was taken on."""
    with open(os.path.join(bench.ROOT, 'profiles', name)) as f:
        d = json.load(f)
    for e in (d.values() if name == 'traffic.json' else [d]):
        assert len(e['source_sha']) == 16 and len(e['source_commit']) >= 7
