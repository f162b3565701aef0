"""GB300 (sm_103a) ONNX RNN / GRU / LSTM sequence operator, and the state
space and token score operators of recurrent language models.

The operators live in a CUDA library with a C ABI (include/onnx_recurrent.h);
``rnn`` and ``ssm`` are its ctypes bindings and ``synth`` draws seeded
synthetic inputs.
"""
from ._build import build
from .rnn import (Plan, RNNError, Stack, rnn_stack_create, rnn_stack_destroy, rnn_stack_last_launch_count,
                  rnn_stack_last_wavefront, rnn_stack_run, rnn_stack_set_wavefront, load, rnn_cell_plan_create, rnn_cell_run, rnn_last_error, rnn_plan_create, rnn_plan_debug_barrier,
                  rnn_plan_destroy, rnn_plan_get_activation, rnn_plan_get_launch,
                  rnn_plan_last_launch_count, rnn_plan_last_timing, rnn_plan_set_launch,
                  rnn_plan_timing_totals,
                  rnn_plan_set_io_type, rnn_plan_set_mode, rnn_plan_set_timing, rnn_plan_set_weights, rnn_plan_sync,
                  rnn_run, run)
from .ssm import (SSM, Scores, rnn_scores, rnn_scores_grad, rnn_ssm_conv, rnn_ssm_conv_grad, rnn_ssm_conv_step,
                  rnn_ssm_create, rnn_ssm_destroy, rnn_ssm_last_launch_count, rnn_ssm_saved_size, rnn_ssm_scan,
                  rnn_ssm_scan_grad, rnn_ssm_scan_step, rnn_ssm_set_io_type, rnn_ssm_sync, scores, scores_grad,
                  ssm_conv, ssm_conv_grad, ssm_scan, ssm_scan_grad)

__all__ = ["build", "load", "Plan", "RNNError", "rnn_plan_create", "rnn_run", "rnn_plan_destroy",
           "rnn_plan_set_mode", "rnn_plan_set_weights", "rnn_plan_sync", "rnn_plan_get_activation",
           "rnn_plan_set_launch", "rnn_plan_get_launch", "rnn_plan_set_timing",
           "rnn_plan_last_timing", "rnn_plan_timing_totals", "rnn_plan_debug_barrier", "rnn_plan_last_launch_count",
           "rnn_last_error", "rnn_cell_plan_create", "rnn_cell_run", "rnn_plan_set_io_type", "Stack", "rnn_stack_create", "rnn_stack_run", "rnn_stack_destroy",
           "rnn_stack_last_launch_count", "rnn_stack_set_wavefront", "rnn_stack_last_wavefront", "run",
           "SSM", "Scores", "rnn_scores", "rnn_scores_grad", "rnn_ssm_conv", "rnn_ssm_conv_grad", "rnn_ssm_conv_step",
           "rnn_ssm_create", "rnn_ssm_destroy", "rnn_ssm_last_launch_count", "rnn_ssm_saved_size", "rnn_ssm_scan",
           "rnn_ssm_scan_grad", "rnn_ssm_scan_step", "rnn_ssm_set_io_type", "rnn_ssm_sync", "scores", "scores_grad",
           "ssm_conv", "ssm_conv_grad", "ssm_scan", "ssm_scan_grad"]
